// span_api.cu -- host side of lite_qk_rope, lite_attn_span and lite_attn_prefix (lite_attn.h).
//
// Validates arguments (before any CUDA call), builds the tensor maps, chooses how the work is split
// and enqueues the kernels.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "host_common.h"
#include "lite_attn.h"
#include "rope_kernel.cuh"
#include "span_kernel.cuh"

namespace {

using lite_host::aligned16;
using lite_host::aligned4;
using lite_host::DeviceContext;

constexpr int kMaxDevices = 64;
constexpr int kRopeMaxRow = 16384;  // elements of a token's row: a block holds a whole token

cudaStream_t as_stream(lite_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------------------------- rotation

// Strides (batch, token, head) of a [B, N, heads, d] tensor: at least `least`, multiples of `unit`
// elements (16 bytes) wherever the dimension has more than one entry.
bool rope_strides_ok(const int64_t* s, int B, int N, int heads, int unit, int least) {
  const int n[3] = {B, N, heads};
  for (int x = 0; x < 3; ++x)
    if (n[x] > 1 && (s[x] < least || s[x] % unit)) return false;
  return true;
}

// Turns per position of angular frequency f; for whole positions its fractional part as a 64-bit
// fraction (in the bits of the double).
double turns_of(double f, bool whole) {
  const long double t = static_cast<long double>(f) / 6.283185307179586476925286766559L;
  if (!whole) return static_cast<double>(t);
  const long double part = t - floorl(t);
  const uint64_t bits = part >= 1.0L ? 0 : static_cast<uint64_t>(part * 18446744073709551616.0L);
  double out;
  std::memcpy(&out, &bits, sizeof(out));
  return out;
}

lite::RopeShape rope_shape(int heads, int d, int U) {
  lite::RopeShape sh;
  sh.units = heads * (d / 16);
  // as many tokens as fit 256 units; a token with more units has a block of its own
  sh.tpb = std::max(1, 256 / std::max(sh.units, 1));
  sh.threads = (sh.tpb * sh.units + U * 32 - 1) / (U * 32) * 32;
  sh.ahead = std::min(8, std::max(1, sh.threads / (sh.tpb * (d / 2))));
  return sh;
}

std::mutex g_rope_mu;

// Sets the dynamic shared memory limit of a rope kernel on the current device, once and to the most that any
// accepted head count takes: the limit is one value for all calls, so a call must never lower it (another
// thread may be about to launch with more).
template <typename T, int D, int U, int NORM, bool ONE>
int rope_smem_limit() {
  static bool set[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LITE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_rope_mu);
  if (set[dev]) return LITE_OK;
  using R = lite::RopeCfg<T, U>;
  size_t most = 0;
  for (int heads = 1; heads * D <= kRopeMaxRow; ++heads)
    most = std::max(most, rope_shape(heads, D, U).bytes(R::STAGES * R::STEP, D, heads));
  if (cudaFuncSetAttribute(lite::lite_rope_kernel<T, D, U, NORM, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(most)) != cudaSuccess)
    return LITE_ERR_CUDA;
  set[dev] = true;
  return LITE_OK;
}

template <typename T, int D, int U, int NORM, bool ONE>
int launch_rope(lite::RopeParams p, const DeviceContext& dc, cudaStream_t stream) {
  const auto kernel = lite::lite_rope_kernel<T, D, U, NORM, ONE>;
  const lite::RopeShape sq = rope_shape(p.t[0].heads, D, U), sk = rope_shape(std::max(p.t[1].heads, 1), D, U);
  const bool keys = p.t[1].heads > 0;
  const int threads = keys ? std::max(sq.threads, sk.threads) : sq.threads;
  using R = lite::RopeCfg<T, U>;
  size_t smem = sq.bytes(R::STAGES * R::STEP, D, p.t[0].heads);
  if (keys) smem = std::max(smem, sk.bytes(R::STAGES * R::STEP, D, p.t[1].heads));
  if (smem > 48 * 1024 && rope_smem_limit<T, D, U, NORM, ONE>() != LITE_OK) return LITE_ERR_CUDA;
  const int64_t need_q = ceil_div(p.tokens, sq.tpb), need_k = keys ? ceil_div(p.tokens, sk.tpb) : 0;
  int64_t q_blocks = need_q, k_blocks = need_k;
  if (need_q + need_k > dc.sms) {
    // persistent: every resident block, shared out by the tensors' work
    int per_sm = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess)
      return LITE_ERR_CUDA;
    const int64_t all = std::max<int64_t>(2, int64_t(dc.sms) * std::max(per_sm, 1));
    if (need_q + need_k > all) {
      const double part = keys ? double(need_q * sq.threads) / double(need_q * sq.threads + need_k * sk.threads) : 1.0;
      q_blocks = std::min(need_q, std::max<int64_t>(1, keys ? std::min<int64_t>(all - 1, int64_t(part * all + 0.5)) : all));
      k_blocks = std::min(need_k, all - q_blocks);
    }
  }
  p.q_blocks = int(q_blocks);
  kernel<<<unsigned(q_blocks + k_blocks), threads, smem, stream>>>(p, sq, sk);
  return cudaGetLastError() == cudaSuccess ? LITE_OK : LITE_ERR_CUDA;
}

template <typename T, int D, int NORM>
int launch_rope_u(const lite::RopeParams& p, const DeviceContext& dc, cudaStream_t stream) {
  // two units a thread: a token of up to 1024 units fits a block
  const bool one = rope_shape(p.t[0].heads, D, 2).tpb == 1 &&
                   (p.t[1].heads == 0 || rope_shape(p.t[1].heads, D, 2).tpb == 1);
  return one ? launch_rope<T, D, 2, NORM, true>(p, dc, stream) : launch_rope<T, D, 2, NORM, false>(p, dc, stream);
}

template <typename T>
int launch_rope_d(const lite::RopeParams& p, const lite_rope_args& a, const DeviceContext& dc, cudaStream_t stream) {
  if (a.d == 64) {
    if (a.norm == 0) return launch_rope_u<T, 64, 0>(p, dc, stream);
    return a.norm == 1 ? launch_rope_u<T, 64, 1>(p, dc, stream) : launch_rope_u<T, 64, 2>(p, dc, stream);
  }
  if (a.norm == 0) return launch_rope_u<T, 128, 0>(p, dc, stream);
  return a.norm == 1 ? launch_rope_u<T, 128, 1>(p, dc, stream) : launch_rope_u<T, 128, 2>(p, dc, stream);
}

// ------------------------------------------------------------------------------------ attention

int tile_for(int d) { return d == 64 ? 64 : (d == 128 ? 128 : 0); }

constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements: tensor maps hold strides below 2^40 bytes

// A token or head stride has to be a positive multiple of 8 elements, a batch stride may be 0 (one
// tensor for all batch entries). Strides of dimensions with one entry are not looked at.
bool attn_strides_ok(const int64_t* s, int B, int N, int heads) {
  const int n[3] = {B, N, heads};
  for (int x = 0; x < 3; ++x)
    if (n[x] > 1 && (s[x] < (x == 0 ? 0 : 8) || s[x] % 8 || s[x] > kMaxStride)) return false;
  return true;
}

cuuint64_t map_stride(int extent, int64_t stride_elements, int d) {
  return extent > 1 ? cuuint64_t(stride_elements) * 2 : cuuint64_t(d) * 2;
}

// K or V [B, N, Hk, d] as the 5-D tensor (64, N, d/64, Hk, B): see make_tmap of the dense call.
bool kv_map(const DeviceContext& dc, CUtensorMap* map, const void* ptr, int B, int N, int Hk, int d, const int64_t* st,
            int rows) {
  const int batches = (B > 1 && st[0] != 0) ? B : 1;
  cuuint64_t dims[5] = {64, cuuint64_t(N), cuuint64_t(d / 64), cuuint64_t(Hk), cuuint64_t(batches)};
  cuuint64_t strides[4] = {map_stride(N, st[1], d), 128, map_stride(Hk, st[2], d), map_stride(batches, st[0], d)};
  cuuint32_t box[5] = {64, cuuint32_t(rows), cuuint32_t(d / 64), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return dc.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q [B, N, Hk * G, d] as (d, G, N, Hk, B): a box holds 64 columns of TN tokens x G heads, which land
// in shared memory as TN * G consecutive 128-byte rows.
bool q_map(const DeviceContext& dc, CUtensorMap* map, const void* ptr, int B, int N, int Hk, int G, int d,
           const int64_t* st, int TN) {
  const int batches = (B > 1 && st[0] != 0) ? B : 1;
  cuuint64_t dims[5] = {cuuint64_t(d), cuuint64_t(G), cuuint64_t(N), cuuint64_t(Hk), cuuint64_t(batches)};
  cuuint64_t strides[4] = {map_stride(G, st[2], d), map_stride(N, st[1], d), map_stride(Hk, st[2] * G, d),
                           map_stride(batches, st[0], d)};
  cuuint32_t box[5] = {64, cuuint32_t(G), cuuint32_t(TN), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return dc.encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_attention(const lite_span_args& a, bool prefix) {
  const int Np = prefix ? a.Np : 0;
  if (!a.q || !a.o) return LITE_ERR_INVALID_ARG;
  if (a.B <= 0 || a.H <= 0 || a.Hk <= 0 || a.Nq <= 0 || a.Nk < 0 || Np < 0 || a.Nk + int64_t(Np) == 0)
    return LITE_ERR_INVALID_ARG;
  if ((a.Nk > 0 && (!a.k || !a.v)) || (Np > 0 && (!a.k_prefix || !a.v_prefix))) return LITE_ERR_INVALID_ARG;
  if (a.H % a.Hk) return LITE_ERR_INVALID_ARG;
  if (std::isnan(a.cap) || a.cap < 0.f || std::isinf(a.cap)) return LITE_ERR_INVALID_ARG;
  if (!a.slopes && (a.q_pos || a.k_pos || a.prefix_pos)) return LITE_ERR_INVALID_ARG;
  // a table for some of the batch entries would be read past its end
  if (a.spans && a.span_batches != 1 && a.span_batches != a.B) return LITE_ERR_INVALID_ARG;
  if ((a.q_pos || a.k_pos) && a.pos_batches != 1 && a.pos_batches != a.B) return LITE_ERR_INVALID_ARG;
  const int t = tile_for(a.d);
  if (!t || a.H / a.Hk > 128) return LITE_ERR_UNSUPPORTED;
  if (!aligned16(a.q) || !aligned16(a.o) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.k_prefix) ||
      !aligned16(a.v_prefix))
    return LITE_ERR_UNSUPPORTED;
  if (!aligned4(a.lse) || !aligned4(a.slopes) || !aligned4(a.q_pos) || !aligned4(a.k_pos) || !aligned4(a.prefix_pos) ||
      (reinterpret_cast<uintptr_t>(a.spans) & 7u))
    return LITE_ERR_UNSUPPORTED;
  if (!attn_strides_ok(a.q_stride, a.B, a.Nq, a.H)) return LITE_ERR_UNSUPPORTED;
  if (a.Nk > 0 && (!attn_strides_ok(a.k_stride, a.B, a.Nk, a.Hk) || !attn_strides_ok(a.v_stride, a.B, a.Nk, a.Hk)))
    return LITE_ERR_UNSUPPORTED;
  if (Np > 0 && (!attn_strides_ok(a.k_prefix_stride, 1, Np, a.Hk) || !attn_strides_ok(a.v_prefix_stride, 1, Np, a.Hk)))
    return LITE_ERR_UNSUPPORTED;
  // 32-bit row and tile arithmetic; positions as 32-bit floats are whole up to 2^24
  const int64_t most = int64_t(1) << 30;
  if (a.Nk > most || Np > most || int64_t(a.B) * a.Nq > most || int64_t(a.B) * a.H > most) return LITE_ERR_UNSUPPORTED;
  if (a.slopes && (int64_t(a.Nk) + Np > (1 << 24) || a.Nq > (1 << 24))) return LITE_ERR_UNSUPPORTED;
  return LITE_OK;
}

// One pass over query tiles (see SpanPass): `units` key heads (times batch entries), each with
// `tokens` tokens against `tiles` key tiles.
struct PassPlan {
  int64_t units = 0, pairs = 0, splits = 1, tiles = 0;
  int TN = 0, F = 1;
  bool one = false;  // one query tile only
  int alt = 0;       // and both softmax groups take it: with F = 4 (which joins them in the CTA), or where there are parts
  int64_t items() const { return units * pairs * splits; }
  // what an item writes where the work is split: one part of 32 rows (F = 4), or one of 128 rows a group
  int per_item() const { return F == 4 ? 1 : 2; }
  int rows() const { return F == 4 ? 32 : 128; }
  int64_t part_floats(int d) const { return items() * per_item() * int64_t(lite::span_part_floats(d, rows())); }
};

struct Plan {
  bool stacked = false;  // a prefix pass over tokens of the whole batch beside the own pass
  PassPlan pre, own;
  bool parts = false;
  double us = 0.0;       // estimated time
  void set_parts() {
    parts = true;
    pre.alt = pre.one;
    own.alt = own.one;
  }
  int64_t part_bytes(int d) const { return parts ? (pre.part_floats(d) + own.part_floats(d)) * int64_t(sizeof(float)) : 0; }
};

constexpr int64_t kMaxPartBytes = int64_t(1) << 30;

PassPlan make_pass(int64_t units, int64_t tokens, int G, int64_t tiles) {
  PassPlan ps;
  ps.units = units;
  ps.tiles = tiles;
  // Up to 32 rows (tokens x grouped heads): four copies of the rows share the key columns (F = 4).
  ps.F = tokens * G <= 32 ? 4 : 1;
  ps.TN = (ps.F == 4 ? 32 : 128) / G;
  const int64_t tq = ceil_div(tokens, ps.TN);
  ps.one = tq == 1;
  ps.alt = ps.one && ps.F == 4;
  ps.pairs = ceil_div(tq, 2);
  return ps;
}

// Microseconds that one CTA takes for an item of t key tiles: its start and end, and each tile, as
// measured on a B200 with few CTAs and with all of them busy (a d = 64 tile has half the keys and shares
// its SM).
double item_us(const PassPlan& ps, int d, double t, bool busy) {
  double tile;
  if (ps.F == 4)
    tile = d == 64 ? (busy ? 1.0 : 0.75) : (busy ? 1.35 : 1.05);
  else if (ps.alt)
    tile = d == 64 ? (busy ? 0.9 : 0.7) : (busy ? 1.4 : 1.1);
  else if (ps.one)  // unsplit, one group takes all tiles (64 rows, 144 heads, 256 tiles, d = 128: 484 us, 396 split in two)
    tile = d == 64 ? (busy ? 1.25 : 1.2) : 1.85;
  else
    tile = d == 64 ? (busy ? 1.75 : 1.25) : (busy ? 2.4 : 2.1);
  return 4.0 + tile * t;
}

// Time of both passes' items on `slots` CTAs: whole waves where all items are alike, else the
// bound of list scheduling. (The spans are on the device: every query tile counts with all keys.)
double plan_us(const Plan& pl, int d, int64_t slots) {
  const int64_t np = pl.pre.items(), no = pl.own.items();
  const bool busy = 2 * (np + no) > slots;
  const double tp = np ? item_us(pl.pre, d, double(ceil_div(pl.pre.tiles, pl.pre.splits)), busy) : 0.0;
  const double to = no ? item_us(pl.own, d, double(ceil_div(pl.own.tiles, pl.own.splits)), busy) : 0.0;
  double us;
  if (np == 0 || no == 0)
    us = double(ceil_div(np + no, slots)) * std::max(tp, to);
  else
    us = std::max(std::max(tp, to), (double(np) * tp + double(no) * to) / double(slots) + to * 0.5);
  if (pl.parts) {
    // the join: its launch, scratch and the parts' way through L2; passes of two kinds take a launch each
    if (pl.part_bytes(d) > kMaxPartBytes) return 1e30;
    us += 8.0 + double(pl.part_bytes(d)) * 2.0 / 4e6 + (np && no && pl.pre.F != pl.own.F ? 4.0 : 0.0);
  }
  return us;
}

// Splits the key ranges where that shortens the plan: few items leave SMs idle, and one long item
// can outlast all others.
void choose_splits(Plan& pl, int d, int64_t slots) {
  pl.us = plan_us(pl, d, slots);
  const Plan base = pl;
  const int64_t longest = std::max(base.pre.tiles, base.own.tiles);
  const int64_t most = std::max<int64_t>(base.pre.items() + base.own.items(), 0) + 4 * slots;
  for (int64_t s = 2; s <= 256 && s <= longest; ++s) {
    Plan c = base;
    const int64_t t = ceil_div(longest, s);
    c.pre.splits = std::max<int64_t>(1, ceil_div(c.pre.tiles, t));
    c.own.splits = std::max<int64_t>(1, ceil_div(c.own.tiles, t));
    c.set_parts();
    if (c.pre.items() + c.own.items() > most) break;
    c.us = plan_us(c, d, slots);
    if (c.us < pl.us) pl = c;
  }
}

Plan make_plan(const lite_span_args& a, int Np, int Tp, int Tk, int64_t slots) {
  const int G = a.H / a.Hk;
  Plan best;
  best.own = make_pass(int64_t(a.B) * a.Hk, a.Nq, G, int64_t(Tp) + Tk);
  choose_splits(best, a.d, slots);
  // Tokens of several entries in one query tile: the batch's tokens have to be evenly spaced in q.
  const bool flat = a.B > 1 && a.q_stride[0] > 0 && (a.Nq == 1 || a.q_stride[0] == int64_t(a.Nq) * a.q_stride[1]);
  if (Np > 0 && flat) {
    Plan c;
    c.stacked = true;
    c.pre = make_pass(a.Hk, int64_t(a.B) * a.Nq, G, Tp);
    if (a.Nk > 0) c.own = make_pass(int64_t(a.B) * a.Hk, a.Nq, G, Tk);
    c.set_parts();
    choose_splits(c, a.d, slots);
    if (c.us < best.us) best = c;
  }
  return best;
}

bool g_span_smem[kMaxDevices][16];
std::mutex g_span_mu;

struct Maps {
  CUtensorMap q, q_stack, k, v, kp, vp;
};

template <int D, int BN, int MOD, int F>
int launch_span(const DeviceContext& dc, const Maps& m, const lite::SpanParams& p, cudaStream_t stream) {
  using C = lite::SpanCfg<D, BN>;
  {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LITE_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_span_mu);
    bool& set = g_span_smem[dev][(D == 128 ? 8 : 0) + (F == 4 ? 4 : 0) + MOD];
    if (!set) {
      if (cudaFuncSetAttribute(lite::lite_span_kernel<D, BN, MOD, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM_BYTES) != cudaSuccess)
        return LITE_ERR_CUDA;
      set = true;
    }
  }
  int64_t grid = int64_t(dc.sms) * C::CTAS_PER_SM;
  if (dc.max_ctas > 0) grid = std::min<int64_t>(grid, dc.max_ctas);
  grid = std::min<int64_t>(grid, p.n_items);
  lite::lite_span_kernel<D, BN, MOD, F>
      <<<unsigned(grid), C::THREADS, C::SMEM_BYTES, stream>>>(m.q, m.q_stack, m.k, m.v, m.kp, m.vp, p);
  return cudaGetLastError() == cudaSuccess ? LITE_OK : LITE_ERR_CUDA;
}

template <int D, int BN, int F>
int launch_span_mod(int mod, const DeviceContext& dc, const Maps& m, const lite::SpanParams& p, cudaStream_t stream) {
  switch (mod) {
    case 0: return launch_span<D, BN, 0, F>(dc, m, p, stream);
    case 1: return launch_span<D, BN, 1, F>(dc, m, p, stream);
    case 2: return launch_span<D, BN, 2, F>(dc, m, p, stream);
    default: return launch_span<D, BN, 3, F>(dc, m, p, stream);
  }
}

int launch_span_any(int d, int F, int mod, const DeviceContext& dc, const Maps& m, const lite::SpanParams& p,
                    cudaStream_t stream) {
  if (d == 64)
    return F == 4 ? launch_span_mod<64, 64, 4>(mod, dc, m, p, stream) : launch_span_mod<64, 64, 1>(mod, dc, m, p, stream);
  return F == 4 ? launch_span_mod<128, 128, 4>(mod, dc, m, p, stream) : launch_span_mod<128, 128, 1>(mod, dc, m, p, stream);
}

bool make_maps(const lite_span_args& a, int Np, const DeviceContext& dc, const Plan& pl, Maps* m) {
  const int t = tile_for(a.d), G = a.H / a.Hk;
  const int tn = pl.own.items() ? pl.own.TN : pl.pre.TN;
  if (!q_map(dc, &m->q, a.q, a.B, a.Nq, a.Hk, G, a.d, a.q_stride, tn)) return false;
  m->q_stack = m->q;
  if (pl.stacked) {
    const int64_t st[3] = {0, a.Nq > 1 ? a.q_stride[1] : a.q_stride[0], a.q_stride[2]};
    if (!q_map(dc, &m->q_stack, a.q, 1, a.B * a.Nq, a.Hk, G, a.d, st, pl.pre.TN)) return false;
  }
  if (a.Nk > 0 && (!kv_map(dc, &m->k, a.k, a.B, a.Nk, a.Hk, a.d, a.k_stride, t) ||
                   !kv_map(dc, &m->v, a.v, a.B, a.Nk, a.Hk, a.d, a.v_stride, t)))
    return false;
  if (Np > 0 && (!kv_map(dc, &m->kp, a.k_prefix, 1, Np, a.Hk, a.d, a.k_prefix_stride, t) ||
                 !kv_map(dc, &m->vp, a.v_prefix, 1, Np, a.Hk, a.d, a.v_prefix_stride, t)))
    return false;
  // a map without keys is never loaded from
  if (a.Nk == 0) m->k = m->kp, m->v = m->vp;
  if (Np == 0) m->kp = m->k, m->vp = m->v;
  return true;
}

lite::SpanPass kernel_pass(const PassPlan& ps, int64_t part0, int64_t slots) {
  lite::SpanPass k;
  k.items = int(ps.items());
  k.pairs = int(ps.pairs);
  k.splits = int(ps.splits);
  k.alt = ps.alt;
  k.TN = ps.TN;
  k.per_item = ps.per_item();
  k.rows = ps.rows();
  k.part0 = part0;
  k.tail = int(std::min(ps.units, ceil_div(2 * slots, std::max<int64_t>(ps.pairs * ps.splits, 1))));
  return k;
}

int run_span(const lite_span_args& a, bool prefix, cudaStream_t stream) {
  const int Np = prefix ? a.Np : 0;
  DeviceContext dc;
  if (lite_host::device_context(false, &dc) != LITE_OK) return LITE_ERR_CUDA;
  const int t = tile_for(a.d);
  const int64_t slots = int64_t(dc.sms) * (a.d == 64 ? 2 : 1);
  const int Tp = int(ceil_div(Np, t));
  const Plan pl = make_plan(a, Np, Tp, int(ceil_div(a.Nk, t)), slots);
  const int64_t items = pl.pre.items() + pl.own.items();
  if (items > INT_MAX / 2) return LITE_ERR_UNSUPPORTED;
  lite::SpanParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = a.B;
  p.H = a.H;
  p.Hk = a.Hk;
  p.G = a.H / a.Hk;
  p.Nq = a.Nq;
  p.Nk = a.Nk;
  p.Np = Np;
  p.Tp = Tp;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.v_stride[0] = a.B > 1 ? a.v_stride[0] : 0;
  p.v_stride[1] = a.Nk > 1 ? a.v_stride[1] : 0;
  p.v_stride[2] = a.Hk > 1 ? a.v_stride[2] : 0;
  p.spans = a.spans;
  p.span_b = a.span_batches > 1 ? 2ll * a.Nq : 0;
  p.slopes = a.slopes;
  p.q_pos = a.q_pos;
  p.k_pos = a.k_pos;
  p.p_pos = a.prefix_pos;
  p.q_pos_b = a.pos_batches > 1 ? a.Nq : 0;
  p.k_pos_b = a.pos_batches > 1 ? a.Nk : 0;
  p.status = dc.status;
  p.wait_limit_ns = dc.wait_limit_ns;
  p.debug_stall = dc.debug_stall;
  p.q_bm = a.B > 1 && a.q_stride[0] != 0;
  p.k_bm = a.B > 1 && a.k_stride[0] != 0;
  p.v_bm = a.B > 1 && a.v_stride[0] != 0;
  p.fused = !pl.stacked;
  p.pre = kernel_pass(pl.pre, 0, slots);
  p.own = kernel_pass(pl.own, pl.pre.part_floats(a.d), slots);
  const float scale = (a.scale > 0.f && !std::isnan(a.scale)) ? a.scale : 1.0f / std::sqrt(float(a.d));
  p.scale_log2 = scale * 1.4426950408889634f;
  if (a.cap > 0.f) {
    p.cap_a = std::min(2.f * p.scale_log2 / a.cap, 3e38f);
    p.cap_c = a.cap * 1.4426950408889634f;
    // tanh(z) / z on |z| <= 0.6 as a polynomial in z^2: the least largest relative error (7.3e-8) of
    // degree 4, fitted numerically; z = s scale / cap
    const double c[5] = {0.999999927, -0.3333231, 0.133101736, -0.0521014795, 0.0154754266};
    const double zs = double(scale) / a.cap;
    if (zs > 1e4) {
      // a cap next to nothing: its coefficients would leave the 32-bit range, and the other form is as exact
      p.cap_mid = p.cap_near = -1.f;
    } else {
      p.cap_mid = float(0.6 / zs);
      // (and not so large that a row's reference, the largest |score|, is far from its maximum: 24 in log2 units)
      p.cap_near = float(std::min(0.6 / zs, 24.0 / (double(scale) * 1.4426950408889634)));
      double f = double(scale) * 1.4426950408889634;
      for (int x = 0; x < 5; ++x, f *= zs * zs) p.cap_b[x] = float(c[x] * f);
    }
  }
  // Scratch: work counters where there are more items than CTAs (their lengths depend on the spans), and
  // the parts.
  const bool counter = items > slots;
  const size_t bytes = (counter ? 256 : 0) + size_t(pl.part_bytes(a.d));
  Maps m;
  if (!make_maps(a, Np, dc, pl, &m)) return LITE_ERR_CUDA;
  char* ws = nullptr;
  if (bytes) {
    if (lite_host::device_context(true, &dc) != LITE_OK) return LITE_ERR_CUDA;
    if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), bytes, dc.pool, stream) != cudaSuccess) return LITE_ERR_CUDA;
  }
  int st = LITE_OK;
  if (counter) {
    p.work_counter = reinterpret_cast<int*>(ws);
    if (cudaMemsetAsync(ws, 0, 2 * sizeof(int), stream) != cudaSuccess) st = LITE_ERR_CUDA;
  }
  if (pl.parts) p.part = reinterpret_cast<float*>(ws + (counter ? 256 : 0));
  const int mod = (a.cap > 0.f ? lite::kSpanCap : 0) | (a.slopes ? lite::kSpanBias : 0);
  // passes of one kind share a launch
  const bool two = p.pre.items && p.own.items && pl.pre.F != pl.own.F;
  if (!st) {
    lite::SpanParams l = p;
    if (two) l.own.items = 0;
    l.n_items = l.pre.items + l.own.items;
    st = launch_span_any(a.d, p.pre.items ? pl.pre.F : pl.own.F, mod, dc, m, l, stream);
  }
  if (!st && two) {
    lite::SpanParams l = p;
    l.pre.items = 0;
    l.n_items = l.own.items;
    if (counter) l.work_counter = p.work_counter + 1;
    st = launch_span_any(a.d, pl.own.F, mod, dc, m, l, stream);
  }
  if (!st && pl.parts) {
    const int64_t threads = int64_t(a.B) * a.Nq * a.H * (a.d / 4);
    const unsigned blocks = unsigned(ceil_div(threads, 256));
    // The join may start once the last CTA of the kernel before has ended, and waits itself until that kernel's
    // writes can be read: without the gap between dependent launches, 2 us less (20.5 against 22.5 us for a tiny call).
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    std::memset(&attr, 0, sizeof(attr));
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, a.d == 64 ? lite::lite_span_combine_kernel<64> : lite::lite_span_combine_kernel<128>,
                           p) != cudaSuccess)
      st = LITE_ERR_CUDA;
  }
  if (ws && cudaFreeAsync(ws, stream) != cudaSuccess && !st) st = LITE_ERR_CUDA;
  return st;
}

}  // namespace

extern "C" {

int lite_qk_rope(const lite_rope_args* args, lite_stream_t stream) {
  if (!args) return LITE_ERR_INVALID_ARG;
  const lite_rope_args& a = *args;
  const bool keys = a.k != nullptr;
  if (!a.q || !a.q_out || (keys && !a.k_out) || !a.freq || !a.axis) return LITE_ERR_INVALID_ARG;
  if (a.B <= 0 || a.N <= 0 || a.H <= 0 || (keys && a.Hk <= 0)) return LITE_ERR_INVALID_ARG;
  if (a.dtype < LITE_BF16 || a.dtype > LITE_FP32 || (a.pairing != 0 && a.pairing != 1) || a.norm < 0 || a.norm > 2)
    return LITE_ERR_INVALID_ARG;
  if (a.norm && (!a.q_weight || (keys && !a.k_weight) || !(a.eps >= 0.f) || std::isinf(a.eps))) return LITE_ERR_INVALID_ARG;
  if (a.n_axes < 1 || a.n_axes > lite::kRopeMaxAxes) return LITE_ERR_INVALID_ARG;
  if (a.d != 64 && a.d != 128) return LITE_ERR_UNSUPPORTED;
  for (int x = 0; x < a.d / 2; ++x)
    if (a.axis[x] < 0 || a.axis[x] >= a.n_axes || !std::isfinite(a.freq[x])) return LITE_ERR_INVALID_ARG;
  if (!a.pos) {
    // the tokens start .. start + N - 1 have to lie in the grid
    if (!a.grid || a.start < 0) return LITE_ERR_INVALID_ARG;
    long double cells = 1;
    for (int x = 0; x < a.n_axes; ++x) {
      if (a.grid[x] <= 0) return LITE_ERR_INVALID_ARG;
      cells *= a.grid[x];
    }
    if (a.start > INT64_MAX - a.N || static_cast<long double>(a.start) + a.N > cells) return LITE_ERR_INVALID_ARG;
  } else if (a.pos_dtype != LITE_FP32 && a.pos_dtype != LITE_INT32) {
    return LITE_ERR_INVALID_ARG;
  } else if (a.pos_batch_stride < 0 || a.pos_axis_stride < 0) {
    return LITE_ERR_INVALID_ARG;
  }
  const int unit = a.dtype == LITE_FP32 ? 4 : 8;
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.q_out) || !aligned16(a.k_out) || !aligned16(a.q_weight) ||
      !aligned16(a.k_weight) || !aligned4(a.pos))
    return LITE_ERR_UNSUPPORTED;
  // (an output stride of 0 would have several rows written to one place)
  if (!rope_strides_ok(a.q_stride, a.B, a.N, a.H, unit, 0) || !rope_strides_ok(a.q_out_stride, a.B, a.N, a.H, 8, 8))
    return LITE_ERR_UNSUPPORTED;
  if (keys && (!rope_strides_ok(a.k_stride, a.B, a.N, a.Hk, unit, 0) ||
               !rope_strides_ok(a.k_out_stride, a.B, a.N, a.Hk, 8, 8)))
    return LITE_ERR_UNSUPPORTED;
  // a block holds a whole token, two units of 16 elements a thread
  if (int64_t(a.H) * a.d > kRopeMaxRow || (keys && int64_t(a.Hk) * a.d > kRopeMaxRow) || int64_t(a.B) * a.N > (1 << 30))
    return LITE_ERR_UNSUPPORTED;
  DeviceContext dc;
  if (lite_host::device_context(false, &dc) != LITE_OK) return LITE_ERR_CUDA;
  lite::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  const auto fill = [](lite::RopeTensor& t, const void* x, void* y, const float* w, const int64_t* xs, const int64_t* ys,
                       int heads) {
    t.x = x;
    t.y = static_cast<__nv_bfloat16*>(y);
    t.w = w;
    for (int i = 0; i < 3; ++i) {
      t.xs[i] = xs[i];
      t.ys[i] = ys[i];
    }
    t.heads = heads;
  };
  fill(p.t[0], a.q, a.q_out, a.q_weight, a.q_stride, a.q_out_stride, a.H);
  if (keys) fill(p.t[1], a.k, a.k_out, a.k_weight, a.k_stride, a.k_out_stride, a.Hk);
  p.tokens = a.B * a.N;
  p.N = a.N;
  p.n_magic = (uint64_t(1) << 63) / uint64_t(a.N) + 1;
  p.halves = a.pairing;
  p.eps = a.eps;
  p.n_axes = a.n_axes;
  p.start = a.start;
  if (!a.pos)
    for (int x = 0; x < a.n_axes; ++x) p.grid[x] = a.grid[x];
  p.pos = a.pos;
  p.pos_is_int = a.pos_dtype == LITE_INT32;
  p.pos_b = a.pos_batch_stride;
  p.pos_a = a.pos_axis_stride;
  p.whole = !a.pos || p.pos_is_int;
  for (int x = 0; x < a.d / 2; ++x) {
    p.turns[x] = turns_of(a.freq[x], p.whole);
    p.axis[x] = uint8_t(a.axis[x]);
  }
  switch (a.dtype) {
    case LITE_BF16: return launch_rope_d<__nv_bfloat16>(p, a, dc, as_stream(stream));
    case LITE_FP16: return launch_rope_d<__half>(p, a, dc, as_stream(stream));
    default: return launch_rope_d<float>(p, a, dc, as_stream(stream));
  }
}

int lite_attn_span(const lite_span_args* args, lite_stream_t stream) {
  if (!args) return LITE_ERR_INVALID_ARG;
  const int st = check_attention(*args, false);
  return st ? st : run_span(*args, false, as_stream(stream));
}

int lite_attn_prefix(const lite_span_args* args, lite_stream_t stream) {
  if (!args) return LITE_ERR_INVALID_ARG;
  const int st = check_attention(*args, true);
  return st ? st : run_span(*args, true, as_stream(stream));
}

}  // extern "C"
