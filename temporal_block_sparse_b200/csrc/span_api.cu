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

cudaStream_t as_stream(lite_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// ------------------------------------------------------------------------------------- rotation

// Strides (batch, token, head) of a [B, N, heads, d] tensor: non-negative, multiples of `unit`
// elements (16 bytes) wherever the dimension has more than one entry.
bool rope_strides_ok(const int64_t* s, int B, int N, int heads, int unit) {
  const int n[3] = {B, N, heads};
  for (int x = 0; x < 3; ++x)
    if (n[x] > 1 && (s[x] < 0 || s[x] % unit)) return false;
  return true;
}

template <typename T, int D, bool HALVES>
int launch_rope(const lite::RopeParams& p0, cudaStream_t stream) {
  lite::RopeParams p = p0;
  constexpr int U = 2;  // units of a thread
  // tokens per block: as many as fit 512 units; a token with more units has a block of its own
  p.tpb = std::max(1, 512 / p.units);
  const int threads = (p.tpb * p.units + U * 32 - 1) / (U * 32) * 32;
  const long long blocks = (static_cast<long long>(p.tokens) + p.tpb - 1) / p.tpb;
  const int heads = p.t[0].heads + p.t[1].heads;
  const size_t smem = size_t(p.tpb) * (D + heads + 2) * sizeof(float);
  lite::lite_rope_kernel<T, D, HALVES, U><<<unsigned(blocks), threads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? LITE_OK : LITE_ERR_CUDA;
}

template <typename T>
int launch_rope_d(const lite::RopeParams& p, int d, int pairing, cudaStream_t stream) {
  if (d == 64) return pairing ? launch_rope<T, 64, true>(p, stream) : launch_rope<T, 64, false>(p, stream);
  return pairing ? launch_rope<T, 128, true>(p, stream) : launch_rope<T, 128, false>(p, stream);
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

// How the work is split into items.
struct Plan {
  bool stacked;              // a prefix pass over tokens of the whole batch, then the own pass
  int pre_pairs, pre_splits, own_pairs, own_splits;
  int64_t n_items;
  bool parts;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Plan make_plan(const lite_span_args& a, int Np, int TN, int Tp, int Tk, int64_t slots) {
  Plan pl;
  std::memset(&pl, 0, sizeof(pl));
  const int64_t tq_own = ceil_div(a.Nq, TN), tq_pre = ceil_div(int64_t(a.B) * a.Nq, TN);
  const bool flat = a.B == 1 || a.Nq == 1 || a.q_stride[0] == int64_t(a.Nq) * a.q_stride[1];
  // Stacking the batch's tokens into common tiles pays where it saves a quarter of the prefix pass
  // or more; it costs a second pass over the parts.
  pl.stacked = Np > 0 && a.B > 1 && flat && a.q_stride[0] > 0 && tq_pre * 4 <= a.B * tq_own * 3;
  int64_t items_p = 0, items_o = 0, tiles_o = Tk;
  if (pl.stacked) {
    pl.pre_pairs = int(ceil_div(tq_pre, 2));
    items_p = int64_t(a.Hk) * pl.pre_pairs;
    pl.own_pairs = a.Nk > 0 ? int(ceil_div(tq_own, 2)) : 0;
  } else {
    pl.own_pairs = int(ceil_div(tq_own, 2));
    tiles_o += Tp;
  }
  items_o = int64_t(a.B) * a.Hk * pl.own_pairs;
  pl.pre_splits = pl.own_splits = 1;
  // Few items leave SMs idle: their key ranges are split so that the longest CTA's work (items it
  // takes, each t tiles and about two more for its start and its end) is shortest.
  if (items_p + items_o < slots) {
    const int64_t longest = std::max<int64_t>(pl.stacked ? Tp : 0, items_o ? tiles_o : 0);
    int64_t best = INT64_MAX;
    for (int64_t s = 1; s <= 128 && s <= longest; ++s) {
      const int64_t t = ceil_div(longest, s);
      const int64_t sp = items_p ? ceil_div(Tp, t) : 1, so = items_o ? std::max<int64_t>(1, ceil_div(tiles_o, t)) : 1;
      const int64_t n = items_p * sp + items_o * so;
      if (n > 2 * slots) break;
      const int64_t cost = ceil_div(n, slots) * (t + 2) + ((sp > 1 || so > 1 || pl.stacked) ? 3 : 0);
      if (cost < best) {
        best = cost;
        pl.pre_splits = int(sp);
        pl.own_splits = int(so);
      }
    }
  }
  pl.n_items = items_p * pl.pre_splits + items_o * pl.own_splits;
  pl.parts = pl.stacked || pl.own_splits > 1;
  return pl;
}

bool g_span_smem[kMaxDevices][8];
std::mutex g_span_mu;

template <int D, int BN, int MOD>
int launch_span(const lite_span_args& a, int Np, const DeviceContext& dc, lite::SpanParams p, const Plan& pl,
                cudaStream_t stream) {
  using C = lite::SpanCfg<D, BN>;
  {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return LITE_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_span_mu);
    bool& set = g_span_smem[dev][(D == 128 ? 4 : 0) + MOD];
    if (!set) {
      if (cudaFuncSetAttribute(lite::lite_span_kernel<D, BN, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM_BYTES) != cudaSuccess)
        return LITE_ERR_CUDA;
      set = true;
    }
  }
  CUtensorMap tq, tqp, tk, tv, tkp, tvp;
  if (!q_map(dc, &tq, a.q, a.B, a.Nq, a.Hk, p.G, D, a.q_stride, p.TN)) return LITE_ERR_CUDA;
  tqp = tq;
  if (pl.stacked) {
    int64_t st[3] = {0, a.Nq > 1 ? a.q_stride[1] : a.q_stride[0], a.q_stride[2]};
    if (!q_map(dc, &tqp, a.q, 1, a.B * a.Nq, a.Hk, p.G, D, st, p.TN)) return LITE_ERR_CUDA;
  }
  if (a.Nk > 0 && (!kv_map(dc, &tk, a.k, a.B, a.Nk, a.Hk, D, a.k_stride, BN) ||
                   !kv_map(dc, &tv, a.v, a.B, a.Nk, a.Hk, D, a.v_stride, BN)))
    return LITE_ERR_CUDA;
  if (Np > 0 && (!kv_map(dc, &tkp, a.k_prefix, 1, Np, a.Hk, D, a.k_prefix_stride, BN) ||
                 !kv_map(dc, &tvp, a.v_prefix, 1, Np, a.Hk, D, a.v_prefix_stride, BN)))
    return LITE_ERR_CUDA;
  if (a.Nk == 0) tk = tkp, tv = tvp;  // never loaded from
  if (Np == 0) tkp = tk, tvp = tv;
  int64_t grid = int64_t(dc.sms) * C::CTAS_PER_SM;
  if (dc.max_ctas > 0) grid = std::min<int64_t>(grid, dc.max_ctas);
  grid = std::min(grid, pl.n_items);
  lite::lite_span_kernel<D, BN, MOD>
      <<<unsigned(grid), C::THREADS, C::SMEM_BYTES, stream>>>(tq, tqp, tk, tv, tkp, tvp, p);
  if (cudaGetLastError() != cudaSuccess) return LITE_ERR_CUDA;
  if (pl.parts) {
    const int64_t threads = int64_t(a.B) * a.Nq * a.H * (D / 4);
    lite::lite_span_combine_kernel<D><<<unsigned(ceil_div(threads, 256)), 256, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return LITE_ERR_CUDA;
  }
  return LITE_OK;
}

template <int D, int BN>
int launch_span_mod(const lite_span_args& a, int Np, const DeviceContext& dc, const lite::SpanParams& p, const Plan& pl,
                    cudaStream_t stream) {
  switch ((a.cap > 0.f ? lite::kSpanCap : 0) | (a.slopes ? lite::kSpanBias : 0)) {
    case 0: return launch_span<D, BN, 0>(a, Np, dc, p, pl, stream);
    case 1: return launch_span<D, BN, 1>(a, Np, dc, p, pl, stream);
    case 2: return launch_span<D, BN, 2>(a, Np, dc, p, pl, stream);
    default: return launch_span<D, BN, 3>(a, Np, dc, p, pl, stream);
  }
}

int run_span(const lite_span_args& a, bool prefix, cudaStream_t stream) {
  const int Np = prefix ? a.Np : 0;
  DeviceContext dc;
  if (lite_host::device_context(false, &dc) != LITE_OK) return LITE_ERR_CUDA;
  const int t = tile_for(a.d);
  lite::SpanParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = a.B;
  p.H = a.H;
  p.Hk = a.Hk;
  p.G = a.H / a.Hk;
  p.Nq = a.Nq;
  p.Nk = a.Nk;
  p.Np = Np;
  p.TN = 128 / p.G;
  p.Tp = int(ceil_div(Np, t));
  const int64_t slots = int64_t(dc.sms) * (a.d == 64 ? 2 : 1);
  const Plan pl = make_plan(a, Np, p.TN, p.Tp, int(ceil_div(a.Nk, t)), slots);
  if (pl.n_items > INT_MAX) return LITE_ERR_UNSUPPORTED;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
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
  p.pre_pairs = pl.pre_pairs;
  p.pre_splits = pl.pre_splits;
  p.own_pairs = pl.own_pairs;
  p.own_splits = pl.own_splits;
  p.pre_items = a.Hk * pl.pre_pairs * pl.pre_splits;
  p.n_items = int(pl.n_items);
  const float scale = (a.scale > 0.f && !std::isnan(a.scale)) ? a.scale : 1.0f / std::sqrt(float(a.d));
  p.scale_log2 = scale * 1.4426950408889634f;
  if (a.cap > 0.f) {
    p.cap_a = 2.f * p.scale_log2 / a.cap;
    p.cap_c = a.cap * 1.4426950408889634f;
  }
  // Scratch: a work counter where items of unequal length are handed out one by one, and the parts.
  const bool counter = a.spans && pl.n_items > slots;
  const size_t floats = a.d == 64 ? lite::SpanPart<64>::FLOATS : lite::SpanPart<128>::FLOATS;
  const size_t bytes = (counter ? 256 : 0) + (pl.parts ? size_t(pl.n_items) * 2 * floats * sizeof(float) : 0);
  char* ws = nullptr;
  if (bytes) {
    if (lite_host::device_context(true, &dc) != LITE_OK) return LITE_ERR_CUDA;
    if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), bytes, dc.pool, stream) != cudaSuccess) return LITE_ERR_CUDA;
  }
  int st = LITE_OK;
  if (counter) {
    p.work_counter = reinterpret_cast<int*>(ws);
    if (cudaMemsetAsync(ws, 0, sizeof(int), stream) != cudaSuccess) st = LITE_ERR_CUDA;
  }
  if (pl.parts) p.part = reinterpret_cast<float*>(ws + (counter ? 256 : 0));
  if (!st)
    st = a.d == 64 ? launch_span_mod<64, 64>(a, Np, dc, p, pl, stream) : launch_span_mod<128, 128>(a, Np, dc, p, pl, stream);
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
  if (!rope_strides_ok(a.q_stride, a.B, a.N, a.H, unit) || !rope_strides_ok(a.q_out_stride, a.B, a.N, a.H, 8))
    return LITE_ERR_UNSUPPORTED;
  if (keys && (!rope_strides_ok(a.k_stride, a.B, a.N, a.Hk, unit) || !rope_strides_ok(a.k_out_stride, a.B, a.N, a.Hk, 8)))
    return LITE_ERR_UNSUPPORTED;
  // a block holds a whole token, two units of 16 elements a thread
  const int64_t units = (int64_t(a.H) + (keys ? a.Hk : 0)) * (a.d / 16);
  if (units > 2048 || int64_t(a.B) * a.N > INT_MAX - 1024) return LITE_ERR_UNSUPPORTED;
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
  p.units = int(units);
  p.units_q = a.H * (a.d / 16);
  p.norm = a.norm;
  p.eps = a.eps;
  p.n_axes = a.n_axes;
  p.start = a.start;
  if (!a.pos)
    for (int x = 0; x < a.n_axes; ++x) p.grid[x] = a.grid[x];
  p.pos = a.pos;
  p.pos_is_int = a.pos_dtype == LITE_INT32;
  p.pos_b = a.pos_batch_stride;
  p.pos_a = a.pos_axis_stride;
  for (int x = 0; x < a.d / 2; ++x) {
    p.turns[x] = a.freq[x] / 6.283185307179586476925;
    p.axis[x] = uint8_t(a.axis[x]);
  }
  switch (a.dtype) {
    case LITE_BF16: return launch_rope_d<__nv_bfloat16>(p, a.d, a.pairing, as_stream(stream));
    case LITE_FP16: return launch_rope_d<__half>(p, a.d, a.pairing, as_stream(stream));
    default: return launch_rope_d<float>(p, a.d, a.pairing, as_stream(stream));
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
