// span_kernel.cuh -- attention in which every query row sees one interval ("span") of keys, for
// sm_100a (tcgen05 + TMEM + TMA): documents packed into one sequence, prefixes, frame-causal and
// windowed rows, padded batches; optionally with scores capped by a tanh, a bias that grows with
// distance, grouped key heads, and a prefix of keys that the whole batch shares.
//
// For query row n of batch entry b and head h, over the Np shared prefix keys and over the keys
// m in [start(n), end(n)) of entry b:
//   s = scale q.k;  s <- cap tanh(s / cap);  s <- s - slope_h |position(n) - position(m)|
//   o = softmax(s) v,  lse = ln sum exp(s);  a row that sees no key has o = 0, lse = -inf.
//
// Rows of a query tile. The MMA takes 128 query rows against one K tile. With grouped heads (G
// query heads per key head) a tile stacks TN = 128 / G tokens x G heads, so a key tile is read once
// for all heads that share it. For a shared prefix and few tokens a sequence, a tile stacks
// tokens of different batch entries (the prefix pass takes the batch as one row of B * Nq tokens),
// so the prefix is read once for the batch.
//
// Up to 32 rows (F = 4) leave three quarters of the MMA's rows empty: they are loaded four times, into
// the lanes of all four warps of a softmax group, and each warp takes a fourth of the tile's key
// columns. Where there is one query tile only, both softmax groups take it, on alternate key
// tiles (`alt`), and this tile's QK^T is issued before the product of the other group's tile. With F = 4
// the eight partial results of a row are joined in the CTA. One token of 8 sequences of up to 32760
// keys (40 heads over 8, d = 128, 839 MB): 249 us with one group and one warp at work, 161-170 us so.
//
// Work items. An item is a pair of query tiles (one per softmax warpgroup), or one tile (alt), and a
// part of the key tiles they see: [prefix tiles][own tiles lo .. hi), of which split s of S takes its
// share. With S = 1 and one pass the item writes o and lse; otherwise it writes its unnormalised O, its
// exponents' reference and its row sum (32-bit) to scratch, and lite_span_combine_kernel joins the
// parts in index order.
//
// Warp roles (320 threads), barriers and the S -> P -> PV chain are those of lite_attn_kernel
// (attn_kernel.cuh): warp 0 finds the key range of the item's rows and feeds K and V by TMA, warp 1
// issues the MMAs, warps 2-5 and 6-9 run the softmax of one query tile each, P staying in TMEM.
// A key tile that every row of the query tile sees entirely takes no mask instruction.
//
// What bounds it. Long rows: the S -> P -> PV -> QK chain of each query tile, as in lite_attn_kernel
// (frame-causal 480p layer, 40 heads, d = 128: 11.3-11.6 ms, 1000 TFLOP/s; tensor pipe 47% busy, exponential
// unit 48%, issue slots 34%). d = 64: issue slots (55%) before the exponential unit (38%). Few rows: HBM (839 MB
// in 154 us, 5.5 TB/s, and the join). Small calls: the chain of key tiles of an item, and the host's call
// (60 items of ten key tiles each, d = 64: 16 us on the GPU, 18 us of the host).
//
// Every wait is bounded as in lite_attn_kernel; on expiry the status word is set and the CTA drains.
#pragma once

#include "attn_kernel.cuh"

namespace lite {

// 1 / x within one unit in the last place (0 for an infinite x)
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(|a|, |b|, |c|)
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
  float y;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

constexpr int kSpanCap = 1, kSpanBias = 2;  // MOD bits of the kernel

// Biases up to this (log2 units) are kept out of the scores exactly. A row's reference is a 32-bit number of the
// bias's size, so it meets the row's maximum within a few units in its last place: 8 here, far from the
// ends of 2^x. Beyond, a score and its bias are one 32-bit sum.
constexpr float kSpanFarBias = 67108864.f;  // 2^26

// One pass over query tiles: the prefix pass (tokens of the whole batch against the shared prefix) or
// the own pass (tokens of one batch entry against its keys).
struct SpanPass {
  int items;                // units * pairs * splits in this launch (units: Hk or B * Hk)
  int pairs;                // work units of query tiles: pairs of tiles, or single tiles (alt)
  int splits;               // parts of the key range
  int alt;                  // both softmax groups take the one query tile, alternate key tiles
  int TN;                   // tokens of a query tile: 128 / G, or 32 / G (F = 4)
  int per_item;             // parts an item writes: 1 (F = 4) or 2
  int rows;                 // rows of a part: 128, or 32 (F = 4)
  long long part0;          // where the pass's parts start in scratch (floats)
  int tail;                 // last units, whose items are handed out together
};

constexpr int kSpanBad = 5;  // key tiles with non-finite values that an item lists

struct SpanParams {
  __nv_bfloat16* o;         // [B, Nq, H, D]
  float* lse;               // [B, H, Nq] or null
  const __nv_bfloat16* v;   // [B, Nk, Hk, D] and its strides (batch, token, head), for the repair of rows
  long long v_stride[3];
  const int* spans;         // [B or 1, Nq, 2] or null (all keys)
  long long span_b;         // 2 * Nq, or 0: one table for all batch entries
  const float* slopes;      // [H] (bias)
  const float* q_pos;       // [B or 1, Nq] or null: Np + Nk - Nq + n
  const float* k_pos;       // [B or 1, Nk] or null: Np + m
  const float* p_pos;       // [Np] or null: m
  long long q_pos_b, k_pos_b;
  float* part;              // scratch of the parts, or null: items write o and lse
  int* work_counter;        // zero before launch; null: static striding over items
  int* status;
  unsigned long long wait_limit_ns;
  int debug_stall;
  int B, H, Hk, G, Nq, Nk, Np;
  int q_bm, k_bm, v_bm;     // 0: the tensor is the same for every batch entry, else 1
  int Tp;                   // prefix key tiles
  int fused;                // own items walk the prefix tiles too
  SpanPass pre, own;
  int n_items;              // pre.items + own.items of this launch
  float scale_log2;         // softmax scale * log2(e)
  float cap_a, cap_c;       // 2 scale log2(e) / cap and cap log2(e)
  float cap_mid;            // the polynomial holds for scores (before scale) up to this: 0.6 cap
  float cap_near;           // and a tile of scores up to this takes the fast path
  float cap_b[5];           // its coefficients in s^2
};

// floats of one part: O of its rows, then the rows' references, then their sums
__host__ __device__ constexpr size_t span_part_floats(int D, int rows) { return size_t(rows) * (D + 2); }

// One query tile of an item. Its key tiles are list entries q = q0, q0 + step, .. (n_live of them): entry
// q < n_pre is prefix tile v_first + q, the others own tile j_first + q - n_pre.
struct SpanTile {
  int tok0;              // its first token (index in the pass: n, or b * Nq + n in the prefix pass)
  int rows;              // valid rows (0: the tile does not exist)
  int n_live, n_pre;
  int j_first;
  int q0, step;
  int full_lo, full_hi;  // every row sees the own keys [full_lo, full_hi)
  // an own tile within [quiet_lo, quiet_hi) is seen entirely by every row of the item that has it (others may be
  // too: span_cuts tells)
  int quiet_lo, quiet_hi;
};

struct SpanInfo {
  int kind;              // -1 end of the work, 0 own pass, 1 prefix pass
  int alt;
  int b, hk;
  int slot;              // index of its first part among the pass's
  int v_first;
  uint32_t u0;           // union index of its first tile
  int n_bad;             // own key tiles whose non-finite values were taken out of shared memory (see
  int bad[kSpanBad];     // span_clean), the first kSpanBad of them by index
  SpanTile t[2];
};

// Place of own key tile j (entry q of its list) among the item's union tiles.
__device__ __forceinline__ int span_union(const SpanInfo& it, int j, int q) {
  if (it.alt) return q;
  const SpanTile& a = it.t[0];
  const SpanTile& b = it.t[1];
  const int na = a.n_live - a.n_pre, nb = b.n_live - b.n_pre;
  const int both = max(0, min(a.j_first + na, b.j_first + nb) - max(a.j_first, b.j_first));
  return max(a.n_pre, b.n_pre) + min(max(j - a.j_first, 0), na) + min(max(j - b.j_first, 0), nb) -
         min(max(j - max(a.j_first, b.j_first), 0), both);
}

struct alignas(8) SpanCtl {
  uint64_t q_full, q_empty;
  uint64_t kv_full[2], kv_free[2];
  uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
  uint64_t item_full[2], item_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  uint32_t ring[4];
  SpanInfo info[2];
};

// The span of a token, clipped to [0, Nk).
__device__ __forceinline__ void span_of(const SpanParams& p, int b, int n, int& s, int& e) {
  s = 0;
  e = p.Nk;
  if (p.spans) {
    const int2 x = __ldg(reinterpret_cast<const int2*>(p.spans + b * p.span_b + 2ll * n));
    s = max(x.x, 0);
    e = min(x.y, p.Nk);
  }
  if (e <= s) s = e = 0;
}

// Decodes item `idx` (whole warp; the result is in every lane).
template <int BN>
__device__ __forceinline__ void span_decode(const SpanParams& p, int idx, int lane, SpanInfo& it) {
  const bool prefix = idx < p.pre.items;
  const SpanPass& ps = prefix ? p.pre : p.own;
  const int i = prefix ? idx : idx - p.pre.items;
  // The last rows first: where rows see their past, these have the most keys. Units one after the other,
  // so that the CTAs at work share keys and values in L2; but the last `tail` units (about two items a
  // CTA) interleaved, for long items started at the very end would keep a few CTAs busy alone.
  const int units = prefix ? p.Hk : p.B * p.Hk, per = ps.pairs * ps.splits;
  int unit = i / per, rem = i - unit * per;
  int rank = rem / ps.splits;
  if (unit >= units - ps.tail) {
    rem = i - (units - ps.tail) * per;
    rank = rem / (ps.tail * ps.splits);
    rem -= rank * (ps.tail * ps.splits);
    unit = units - ps.tail + rem / ps.splits;
  }
  const int split = rem % ps.splits;
  const int pair = ps.pairs - 1 - rank;
  it.kind = prefix ? 1 : 0;
  it.alt = ps.alt;
  it.b = prefix ? 0 : unit / p.Hk;
  it.hk = prefix ? unit : unit - it.b * p.Hk;
  it.slot = ((unit * ps.pairs + rank) * ps.splits + split) * ps.per_item;
  const int ntok = prefix ? p.B * p.Nq : p.Nq;
  const int tp = (prefix || p.fused) ? p.Tp : 0;
  int jlo = 0x7fffffff, jhi = 0;  // own key tiles that either query tile has to see
  int tlo[2] = {0, 0}, thi[2] = {0, 0};  // and each of them
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    SpanTile& t = it.t[g];
    if (ps.alt && g == 1) {
      it.t[1] = it.t[0];
      tlo[1] = tlo[0];
      thi[1] = thi[0];
      break;
    }
    t.tok0 = (ps.alt ? pair : 2 * pair + g) * ps.TN;
    const int toks = max(0, min(ps.TN, ntok - t.tok0));
    t.full_lo = 0;
    t.full_hi = p.Nk;
    t.rows = toks * p.G;
    tlo[g] = thi[g] = 0;
    if (it.kind == 0 && toks > 0) {
      int lo = 0x7fffffff, hi = 0, flo = 0, fhi = p.Nk;
      if (p.spans) {
        for (int x = lane; x < toks; x += 32) {
          int s, e;
          span_of(p, it.b, t.tok0 + x, s, e);
          if (e > s) {
            lo = min(lo, s);
            hi = max(hi, e);
          }
          flo = max(flo, e > s ? s : 0x7fffffff);
          fhi = min(fhi, e);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        flo = __reduce_max_sync(0xffffffffu, flo);
        fhi = __reduce_min_sync(0xffffffffu, fhi);
      } else {
        lo = 0;
        hi = p.Nk;
      }
      if (hi > lo) {
        tlo[g] = lo / BN;
        thi[g] = (hi + BN - 1) / BN;
        jlo = min(jlo, tlo[g]);
        jhi = max(jhi, thi[g]);
      }
      t.full_lo = flo;
      t.full_hi = fhi;
    }
  }
  if (jhi == 0) jlo = 0;
  // virtual tiles: prefix [0, tp), then own jlo .. jhi; this split's are [v0, v1)
  const long long total = tp + (jhi - jlo);
  const int v0 = int(total * split / ps.splits), v1 = int(total * (split + 1) / ps.splits);
  it.v_first = v0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    SpanTile& t = it.t[g];
    t.n_pre = t.rows ? max(0, min(v1, tp) - v0) : 0;
    const int j0 = max(tlo[g], jlo + max(v0 - tp, 0)), j1 = min(thi[g], jlo + v1 - tp);
    t.j_first = j0;
    t.n_live = t.n_pre + (t.rows ? max(0, j1 - j0) : 0);
    t.q0 = ps.alt ? g : 0;
    t.step = ps.alt ? 2 : 1;
    t.quiet_lo = t.full_lo;
    t.quiet_hi = t.full_hi;
  }
  if (ps.alt) {
    it.t[1].n_live >>= 1;
    it.t[0].n_live -= it.t[1].n_live;
    return;
  }
  // where the other query tile has own key tiles that are cut for its rows: those before and behind its full range
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const SpanTile& o = it.t[g ^ 1];
    const int first = o.j_first * BN, end = min((o.j_first + o.n_live - o.n_pre) * BN, p.Nk);
    if (first >= end) continue;
    if (first < o.full_lo) it.t[g].quiet_lo = max(it.t[g].full_lo, o.full_lo);
    if (o.full_hi < end) it.t[g].quiet_hi = min(it.t[g].full_hi, o.full_hi);
  }
}

// Whether some row of query tile t, which has own key tile j, does not see all its keys.
template <int BN>
__device__ __forceinline__ bool span_cuts(const SpanParams& p, const SpanTile& t, int j) {
  return t.full_lo > j * BN || t.full_hi < min(j * BN + BN, p.Nk);
}

// This thread's part of a group's cleaning of own key tile j (entry q of its list): the tile goes into the item's
// list, then its infinities and NaN become 0. Both groups clean a tile that either of them needs clean, each
// before its own product: the products then read the same values whichever group comes first (a weight that
// underflowed to 0 makes NaN of an infinity and 0 of a cleaned one). A group that finds the tile clean
// already finds it in the list too, which is written first; the list brings the values back to the rows
// that see them.
template <typename C, int BN>
__device__ __forceinline__ void span_clean_tile(SpanCtl* ctl, uint8_t* smem, const Waiter& wt, int slot, int tid, int j, int q) {
  SpanInfo& it = ctl->info[slot];
  const uint32_t u = it.u0 + span_union(it, j, q);
  wt.wait(ptx::smem_addr(&ctl->kv_full[(u + 1) & 1]), ((u + 1) >> 1) & 1);  // V_u comes with bundle u + 1
  volatile uint4* const tile = reinterpret_cast<volatile uint4*>(smem + C::OFF_V + (u & 1) * C::KV_BYTES);
  constexpr int PIECES = C::KV_BYTES / 16 / 128;  // 16-byte pieces of a thread
  uint32_t most = 0u;  // largest magnitude of either half-word
#pragma unroll 4
  for (int i = 0; i < PIECES; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(const_cast<const uint4*>(tile + i * 128 + tid));
    most = __vmaxu2(most, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
  }
  if ((most & 0xffffu) >= 0x7f80u || (most >> 16) >= 0x7f80u) {
    int x = 0;
    for (; x < kSpanBad; ++x) {
      const int old = atomicCAS(&it.bad[x], -1, j);
      if (old == -1 || old == j) break;
    }
    atomicMax(&it.n_bad, x + 1);  // kSpanBad + 1: the list is full
    __threadfence_block();
    for (int i = 0; i < PIECES; ++i) {
      volatile uint32_t* const w = reinterpret_cast<volatile uint32_t*>(tile + i * 128 + tid);
      for (int y = 0; y < 4; ++y) {
        uint32_t z = w[y];
        if ((z & 0x7f80u) == 0x7f80u) z &= 0xffff0000u;
        if ((z & 0x7f800000u) == 0x7f800000u) z &= 0xffffu;
        w[y] = z;
      }
    }
  }
  ptx::fence_proxy_async_smem();  // also for what the other group wrote and this thread read
}

// Key r of a tile is at position `at` (NaN: no key): into the tile's positions, and the first and last of each warp's
// keys behind them.
template <int BN>
__device__ __noinline__ void span_publish(float* kp, float at, int r) {
  if (r < BN) kp[r] = at;
  float first = at, last = at;
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    first = fminf(first, __shfl_xor_sync(0xffffffffu, first, x));
    last = fmaxf(last, __shfl_xor_sync(0xffffffffu, last, x));
  }
  if ((r & 31) == 0) *reinterpret_cast<float2*>(kp + BN + r / 16) = make_float2(first, last);
}

// Shared memory: lite_attn_kernel's layout, with a staging area of 32 rows x 128 bytes a softmax warp.
template <int D, int BN>
struct SpanCfg : AttnCfg<D, BN> {
  using A = AttnCfg<D, BN>;
  static constexpr int OST_WARP = 32 * 128;
  static constexpr int SMEM_USED = A::OFF_OST + 8 * OST_WARP + 1024;
  static constexpr int SMEM_BYTES =
      A::CTAS_PER_SM == 2 ? SMEM_USED : (SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024);
  static_assert(A::CTAS_PER_SM == 1 || 2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

constexpr uint32_t kSpanAlt = 2048u;    // ring word: both groups use the first query tile

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// PC (16 or 32) score columns of this lane's row, not yet waited for
template <int PC>
__device__ __forceinline__ void span_load(uint32_t at, float (&v)[PC]) {
  if constexpr (PC == 32)
    ptx::tmem_ld32(at, reinterpret_cast<uint32_t(&)[32]>(v));
  else
    tmem_ld16(at, reinterpret_cast<uint32_t(&)[16]>(v));
}

// four running maxima over the columns, and their maximum
template <int PC>
__device__ __forceinline__ void span_max(const float (&v)[PC], float (&m)[4]) {
#pragma unroll
  for (int x = 0; x < PC; x += 8) {
    m[0] = ptx::fmax3(m[0], v[x], v[x + 1]);
    m[1] = ptx::fmax3(m[1], v[x + 2], v[x + 3]);
    m[2] = ptx::fmax3(m[2], v[x + 4], v[x + 5]);
    m[3] = ptx::fmax3(m[3], v[x + 6], v[x + 7]);
  }
}
__device__ __forceinline__ float span_max4(const float (&m)[4]) { return ptx::fmax3(m[0], m[1], fmaxf(m[2], m[3])); }

// P = 2^exponent of PC columns, in bf16 to TMEM (over score columns that have been read) and summed in acc;
// exponent(x) gives columns x, x + 1
template <int PC, typename E>
__device__ __forceinline__ void span_put(uint32_t at, float2 (&acc)[4], E exponent) {
  uint32_t pk[PC / 2];
#pragma unroll
  for (int x = 0; x < PC / 2; ++x) {
    const float2 a = exponent(2 * x);
    const float2 pp = make_float2(ptx::ex2(a.x), ptx::ex2(a.y));
    acc[x & 3] = __fadd2_rn(acc[x & 3], pp);
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(pp.x, pp.y);
    pk[x] = *reinterpret_cast<const uint32_t*>(&h2);
  }
  if constexpr (PC == 32)
    ptx::tmem_st16(at, pk);
  else
    ptx::tmem_st8(at, pk);
}

// F = 4: the other quarters' key columns of the row are another lane's, P = 0 there
template <int NC>
__device__ __forceinline__ void span_zero(uint32_t s_tmem, int quarter) {
  uint32_t zero[NC / 2];
#pragma unroll
  for (int x = 0; x < NC / 2; ++x) zero[x] = 0u;
#pragma unroll
  for (int c = 1; c < 4; ++c) {
    const uint32_t at = s_tmem + ((quarter + c) & 3) * (NC / 2);
    if constexpr (NC == 32)
      ptx::tmem_st16(at, zero);
    else
      ptx::tmem_st8(at, zero);
  }
}

template <int D>
__device__ __forceinline__ void span_rescale(uint32_t o_tmem, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t rr[32];
    ptx::tmem_ld32(o_tmem + c * 32, rr);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 32; ++x) rr[x] = __float_as_uint(__uint_as_float(rr[x]) * alpha);
    ptx::tmem_st32(o_tmem + c * 32, rr);
  }
}

// A key tile for which the short way does not do (a span ends in it, scores near the cap, rows on both sides of it,
// given positions): every score of the warp's rows in full, back into TMEM, then the exponentials. Keys
// [lo, hi) of this thread's NC columns are seen. Takes and returns (reference, row sum).
//
// Far from its keys a row's bias is much larger than what its scores differ by: at 2^19 log2 units a 32-bit sum of both
// is good to 2^-5. So the least bias among the keys seen (`off`) stays out of the sums: a score is s + (off - bias),
// off - bias one rounding of a small number, and off is taken into account with the reference. At given positions the
// tile's first and last position (of each 32 keys, behind the positions) bound it well enough where they lie within a
// bias of 256 (2^-16); the keys are looked at one by one where not, which takes 20% longer.
template <int D, int NC, int MOD, int F>
__device__ __forceinline__ float2 span_tile_in_full(const SpanParams& p, uint32_t s_tmem, uint32_t o_tmem, int quarter,
                                                 int lo, int hi, float base, float slope, float qp, const float* kpos,
                                                 float2 ml, bool rescale) {
  constexpr bool CAP = (MOD & kSpanCap) != 0, BIAS = (MOD & kSpanBias) != 0;
  constexpr int PC = NC < 32 ? NC : 32;
  const int col0 = F == 1 ? 0 : quarter * NC;
  // the keys seen among columns PC * c .. as bits: one select per column
  const auto seen = [&](int c) -> uint32_t {
    const int a = min(max(lo - PC * c, 0), 32), z = min(max(hi - PC * c, 0), 32);
    const uint32_t upto = z >= 32 ? 0xffffffffu : ((1u << z) - 1u);
    const uint32_t below = a >= 32 ? 0xffffffffu : ((1u << a) - 1u);
    return upto & ~below;
  };
  // column x is lowered by the bias and raised by off: step * |from + x| + rest
  float off = 0.f, step = -slope, from = base, rest = 0.f;
  if constexpr (BIAS) {
    if (kpos) {
      const float4* ends = reinterpret_cast<const float4*>(kpos - col0 + NC * F);
      const float4 e0 = ends[0], e1 = ends[1];
      const float first = fminf(fminf(e0.x, e0.z), fminf(e1.x, e1.z)), last = fmaxf(fmaxf(e0.y, e0.w), fmaxf(e1.y, e1.w));
      float near = fmaxf(fmaxf(first - qp, qp - last), 0.f), far = fmaxf(qp - first, last - qp);
      if (__any_sync(0xffffffffu, fabsf(slope) * (last - first) > 256.f)) {
        near = INFINITY;
        far = 0.f;
#pragma unroll 1
        for (int c = 0; c < NC / PC; ++c) {
          const uint32_t bits = seen(c);
#pragma unroll
          for (int x = 0; x < PC; ++x) {
            const float dist = fabsf(kpos[PC * c + x] - qp);
            near = fminf(near, (bits & (1u << x)) ? dist : INFINITY);
            far = fmaxf(far, (bits & (1u << x)) ? dist : 0.f);
          }
        }
      }
      off = fminf(slope * near, slope * far);
      if (!(fabsf(off) <= kSpanFarBias)) off = 0.f;
      rest = off;
    } else {
      const float a = float(max(lo, 0)), z = float(min(hi, NC) - 1);
      // the least bias is at the first or last of them, or (rows amid the columns) at the row's own position
      const bool one_side = base >= 0.f || base <= 1.f - NC;
      const float end = (base < 0.f) == (slope >= 0.f) ? z : a;
      off = slope * fabsf(base + end);
      if (!one_side)
        off = fminf(fminf(slope * fabsf(base + a), slope * fabsf(base + z)), slope * fabsf(base + fminf(fmaxf(-base, a), z)));
      if (!(fabsf(off) <= kSpanFarBias)) off = 0.f;
      rest = off;
      if (one_side) {
        // the bias grows by |slope| a column from that end, where it is off but for the rounding of off (and of
        // the distance, where that takes more than 24 bits: dist + lost is the sum itself)
        const float dist = base + end, lost = end - (dist - base);
        step = -fabsf(slope);
        from = -end;
        rest = fmaf(dist < 0.f ? slope : -slope, lost, fmaf(-slope, fabsf(dist), off));
      }
    }
  }
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  float v[PC];
#pragma unroll 1
  for (int c = 0; c < NC / PC; ++c) {
    span_load<PC>(s_tmem + col0 + c * PC, v);
    ptx::tmem_wait_ld();
    const uint32_t bits = seen(c);
    const float at = from + float(PC * c);
    const float* kc = kpos + PC * c;
    if constexpr (CAP) {
      float big = 0.f;
#pragma unroll
      for (int x = 0; x < PC; x += 2) big = abs_max3(big, v[x], v[x + 1]);
      const bool all_near = !__any_sync(0xffffffffu, big > p.cap_mid);
#pragma unroll
      for (int x = 0; x < PC; x += 2) {
        const float2 s2 = make_float2(v[x], v[x + 1]);
        const float2 y = __fmul2_rn(s2, s2);
        float2 t = __ffma2_rn(make_float2(p.cap_b[4], p.cap_b[4]), y, make_float2(p.cap_b[3], p.cap_b[3]));
        t = __ffma2_rn(t, y, make_float2(p.cap_b[2], p.cap_b[2]));
        t = __ffma2_rn(t, y, make_float2(p.cap_b[1], p.cap_b[1]));
        t = __ffma2_rn(t, y, make_float2(p.cap_b[0], p.cap_b[0]));
        t = __fmul2_rn(s2, t);
        if (!all_near) {
          // cap tanh(z) = cap - 2 cap / (1 + e^{2z}), in log2 units; both ends saturate exactly. Near zero it
          // cancels (a large cap against small scores), there the polynomial stays.
          const float fx = fmaf(-2.f * p.cap_c, fast_rcp(1.f + ptx::ex2(s2.x * p.cap_a)), p.cap_c);
          const float fy = fmaf(-2.f * p.cap_c, fast_rcp(1.f + ptx::ex2(s2.y * p.cap_a)), p.cap_c);
          t.x = fabsf(s2.x) <= p.cap_mid ? t.x : fx;
          t.y = fabsf(s2.y) <= p.cap_mid ? t.y : fy;
        }
        v[x] = t.x;
        v[x + 1] = t.y;
      }
    } else {
#pragma unroll
      for (int x = 0; x < PC; ++x) v[x] *= p.scale_log2;
    }
#pragma unroll
    for (int x = 0; x < PC; ++x) {
      if (BIAS) v[x] += fmaf(step, fabsf(kpos ? kc[x] - qp : at + float(x)), rest);
      v[x] = (bits & (1u << x)) ? v[x] : -INFINITY;
    }
    span_max<PC>(v, m);
    if constexpr (PC == 32)
      ptx::tmem_st32(s_tmem + col0 + c * 32, reinterpret_cast<uint32_t(&)[32]>(v));
    else
      ptx::tmem_st16(s_tmem + col0, reinterpret_cast<uint32_t(&)[16]>(v));
  }
  ptx::tmem_wait_st();
  const float loc = span_max4(m) - off;
  float m_used = ml.x, l = ml.y, alpha = 1.f;
  const bool need = loc > m_used + kRescaleLog2;
  if (need) {
    alpha = ptx::ex2(m_used - loc);
    m_used = loc;
    l *= alpha;
  }
  const float neg_m = m_used == -INFINITY ? 0.f : -off - m_used;
  const float2 nm2 = make_float2(neg_m, neg_m);
  float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < NC / PC; ++c) {
    span_load<PC>(s_tmem + col0 + c * PC, v);
    ptx::tmem_wait_ld();
    span_put<PC>(s_tmem + col0 / 2 + c * (PC / 2), acc, [&](int x) { return __fadd2_rn(make_float2(v[x], v[x + 1]), nm2); });
  }
  if constexpr (F > 1) span_zero<NC>(s_tmem, quarter);
  if (__any_sync(0xffffffffu, need) && rescale) span_rescale<D>(o_tmem, alpha);
  ptx::tmem_wait_st();
  const float2 acc2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
  return make_float2(m_used, l + acc2.x + acc2.y);
}

// Adds the non-finite values of the keys [ks, ke) that this thread's row sees (columns col0 .. col0 + NC of each
// tile) to its row of O: those of the tiles that were cleaned for the item, as far as they are this group's
// (alternating groups share the list, and when a group reads it the other may not be through).
template <int D, int BN, int NC>
__device__ __forceinline__ void span_repair(const SpanParams& p, const SpanInfo& it, int grp, uint32_t o_tmem, bool valid,
                                         int ks, int ke, int b, int col0) {
  const SpanTile& t = it.t[grp];
  // more tiles than the list holds: all own tiles of the group
  const bool listed = it.n_bad <= kSpanBad;
  const int end = t.j_first + (it.alt ? it.t[0].n_live + it.t[1].n_live : t.n_live) - t.n_pre;
  const int n = listed ? it.n_bad : end - t.j_first;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t rr[32];
    ptx::tmem_ld32(o_tmem + c * 32, rr);
    ptx::tmem_wait_ld();
    for (int x = 0; valid && x < n; ++x) {
      const int j = listed ? it.bad[x] : t.j_first + x;
      if (j < t.j_first || j >= end || (it.alt && ((t.n_pre + j - t.j_first) & 1) != grp)) continue;
      const int m1 = min(ke, j * BN + col0 + NC);
      for (int m = max(ks, j * BN + col0); m < m1; ++m) {
        const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v + b * p.v_stride[0] + m * p.v_stride[1] +
                                                              it.hk * p.v_stride[2] + c * 32);
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const uint32_t w = __ldg(v + y);
          if ((w & 0x7f80u) == 0x7f80u) rr[2 * y] = __float_as_uint(__uint_as_float(rr[2 * y]) + __uint_as_float(w << 16));
          if ((w & 0x7f800000u) == 0x7f800000u)
            rr[2 * y + 1] = __float_as_uint(__uint_as_float(rr[2 * y + 1]) + __uint_as_float(w & 0xffff0000u));
        }
      }
    }
    __syncwarp();
    ptx::tmem_st32(o_tmem + c * 32, rr);
    ptx::tmem_wait_st();
  }
}

template <int D, int BN, int MOD, int F>
__global__ void __launch_bounds__(320, AttnCfg<D, BN>::CTAS_PER_SM)
    lite_span_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQp,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                     const __grid_constant__ SpanParams p) {
  using C = SpanCfg<D, BN>;
  constexpr int NC = BN / F;  // key columns of a thread
  constexpr int PC = NC < 32 ? NC : 32;  // loaded, converted and stored at a time
  constexpr int PR = F == 4 ? 32 : 128;  // rows of a part
  constexpr bool CAP = (MOD & kSpanCap) != 0, BIAS = (MOD & kSpanBias) != 0;
  static_assert(sizeof(SpanCtl) <= C::CTL_BYTES, "control block");
  // key positions of two tiles per warpgroup share the group's staging area
  static_assert((2 * BN + 16) * 4 <= 4 * C::OST_WARP, "position buffer");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  SpanCtl* ctl = reinterpret_cast<SpanCtl*>(smem + C::OFF_CTL);
  const uint32_t sQ = ptx::smem_addr(smem + C::OFF_Q);
  const uint32_t sK = ptx::smem_addr(smem + C::OFF_K);
  const uint32_t sV = ptx::smem_addr(smem + C::OFF_V);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

#define BAR(x) ptx::smem_addr(&ctl->x)

  if (threadIdx.x == 0) {
    ptx::mbar_init(BAR(q_full), 1);
    ptx::mbar_init(BAR(q_empty), 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(BAR(kv_full[b]), 1);
      ptx::mbar_init(BAR(kv_free[b]), 1);
      ptx::mbar_init(BAR(s_full[b]), 1);
      ptx::mbar_init(BAR(p_full[b]), 128);
      ptx::mbar_init(BAR(pv_done[b]), 1);
      ptx::mbar_init(BAR(o_free[b]), 128);
      ptx::mbar_init(BAR(item_full[b]), 1);
      ptx::mbar_init(BAR(item_empty[b]), 8);
    }
    ptx::mbar_init(BAR(drain), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const Waiter wt{&ctl->abort, p.status, p.wait_limit_ns};

  if (warp == 0) {
    // ------------------------------------------------------------------------- TMA producer
    // Bundles as in lite_attn_kernel: bundle u carries K_u and V_{u-1}; kv_free of u-2 frees both
    // stages. The whole warp decodes an item (it reads the spans of the item's tokens), lane 0
    // issues the loads.
    uint32_t u = 0, items = 0, qn = 0;
    bool ok = true;
    bool q_armed = false, kv_armed[2] = {false, false};
    uint32_t q_par = 0, kv_par[2] = {0, 0};
    bool v_needed = false, pv_pre = false;
    int pj = 0, ph = 0, pb = 0;  // V coordinates of union tile u-1
    auto bundle = [&](bool with_k, bool pre, int j, int h, int b, uint32_t flags) -> bool {
      if (u >= 2 && !wt.wait(BAR(kv_free[u & 1]), ((u - 2) >> 1) & 1)) return false;
      ctl->ring[u & 3] = flags;
      const uint32_t bar = BAR(kv_full[u & 1]);
      ptx::mbar_arrive_expect_tx(bar, (with_k ? C::KV_TX : 0u) + (v_needed ? C::KV_TX : 0u));
      if (with_k)
        ptx::tma_load_5d(sK + (u & 1) * C::KV_BYTES, pre ? &tmKp : &tmK, bar, 0, j * BN, 0, h, pre ? 0 : b * p.k_bm);
      if (v_needed)
        ptx::tma_load_5d(sV + ((u - 1) & 1) * C::KV_BYTES, pv_pre ? &tmVp : &tmV, bar, 0, pj * BN, 0, ph,
                         pv_pre ? 0 : pb * p.v_bm);
      v_needed = with_k;
      kv_armed[u & 1] = true;
      kv_par[u & 1] = (u >> 1) & 1;
      pv_pre = pre;
      pj = j;
      ph = h;
      pb = b;
      ++u;
      return true;
    };
    while (true) {
      const int slot = items & 1;
      int item = -1;
      if (lane == 0) {
        if (items >= 2) ok = wt.wait(BAR(item_empty[slot]), ((items >> 1) - 1) & 1);
        if (ok) item = p.work_counter ? atomicAdd(p.work_counter, 1) : int(blockIdx.x + items * gridDim.x);
        if (item >= p.n_items) item = -1;
      }
      ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      if (!ok) break;
      item = __shfl_sync(0xffffffffu, item, 0);
      SpanInfo it;
      it.kind = -1;
      if (item >= 0) span_decode<BN>(p, item, lane, it);
      it.n_bad = 0;
#pragma unroll
      for (int x = 0; x < kSpanBad; ++x) it.bad[x] = -1;
      if (lane == 0) {
        it.u0 = u;
        ctl->info[slot] = it;
        ptx::mbar_arrive(BAR(item_full[slot]));
      }
      ++items;
      if (item < 0) break;
      if (lane == 0) {
        const int n0 = it.t[0].n_live, n1 = it.t[1].n_live;
        if (n0 + n1 == 0) {
          // flush the pending V of the item before, as lite_attn_kernel does for an empty item
          if (v_needed) ok = bundle(false, false, 0, 0, 0, 0u);
        } else {
          if (qn >= 1) ok = wt.wait(BAR(q_empty), (qn - 1) & 1);
          if (ok) {
            // alternating groups share one Q tile; with F = 4 its rows go to all four quarters of it
            const int n_q = it.alt ? 1 : 2;
            const SpanPass& ps = it.kind == 1 ? p.pre : p.own;
            const uint32_t qtx = uint32_t(ps.TN * p.G) * 128u * C::NCHUNK * F;
            ptx::mbar_arrive_expect_tx(BAR(q_full), (n0 > 0 ? qtx : 0u) + (n_q > 1 && n1 > 0 ? qtx : 0u));
            for (int g = 0; g < n_q; ++g)
              if ((g ? n1 : n0) > 0)
                for (int c = 0; c < C::NCHUNK; ++c)
                  for (int x = 0; x < F; ++x)
                    ptx::tma_load_5d(sQ + g * C::Q_BYTES + c * C::Q_CHUNK + x * 4096, it.kind == 1 ? &tmQp : &tmQ,
                                     BAR(q_full), c * 64, 0, it.t[g].tok0, it.hk, it.kind == 1 ? 0 : it.b * p.q_bm);
            q_armed = true;
            q_par = qn & 1;
            const uint32_t item_bits =
                ((qn & 1) ? kItemOdd : 0u) | (qn >= 1 ? kItemAfterFirst : 0u) | (it.alt ? kSpanAlt : 0u);
            uint32_t f = kItemFirst;
            // the union of the two tiles' key tiles: prefix tiles (common to both), then own ones in order
            int d0 = 0, d1 = 0;
            while (ok && (d0 < n0 || d1 < n1)) {
              const int none = 0x7fffffff;
              int c0 = none, c1 = none;
              bool pre;
              if (it.alt) {
                // entries in order, the groups in turn
                const int q = d0 + d1;
                pre = q < it.t[0].n_pre;
                (d0 == d1 ? c0 : c1) = pre ? it.v_first + q : it.t[0].j_first + q - it.t[0].n_pre;
              } else {
                const bool pre0 = d0 < it.t[0].n_pre, pre1 = d1 < it.t[1].n_pre;
                pre = pre0 || pre1;
                if (pre) {
                  if (pre0) c0 = it.v_first + d0;
                  if (pre1) c1 = it.v_first + d1;
                } else {
                  if (d0 < n0) c0 = it.t[0].j_first + d0 - it.t[0].n_pre;
                  if (d1 < n1) c1 = it.t[1].j_first + d1 - it.t[1].n_pre;
                }
              }
              const int j = min(c0, c1);
              f |= item_bits;
              if (c0 == j) {
                f |= kLive0 | (d0 == 0 ? kFirst0 : 0u) | (d0 == n0 - 1 ? kLast0 : 0u);
                ++d0;
              }
              if (c1 == j) {
                f |= kLive1 | (d1 == 0 ? kFirst1 : 0u) | (d1 == n1 - 1 ? kLast1 : 0u);
                ++d1;
              }
              if (d0 == n0 && d1 == n1) f |= kItemLast;
              ok = bundle(true, pre, j, it.hk, it.b, f);
              f = 0u;
            }
            ++qn;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      if (!ok) break;
    }
    if (lane == 0) {
      if (ok) bundle(false, false, 0, 0, 0, kEnd);
      if (q_armed) wt.wait_drain(BAR(q_full), q_par);
      for (int b = 0; b < 2; ++b)
        if (kv_armed[b]) wt.wait_drain(BAR(kv_full[b]), kv_par[b]);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------------- MMA issuer
    // The protocol of lite_attn_kernel: per union tile PV_g(u-1), then QK_g(u), for g = 0, 1.
    if (lane == 0) {
      uint32_t u = 0;
      uint32_t pc[2] = {0, 0};
      uint32_t prev = 0;
      bool ok = true;
      const uint64_t q_desc0 = umma_desc_sw128(sQ, 16, 1024);
      const uint64_t k_desc0 = umma_desc_sw128(sK, 16, 1024);
      const uint64_t v_desc0 = umma_desc_sw128(sV, C::KV_CHUNK, 1024);
      const uint32_t bar_kv = BAR(kv_full[0]), bar_free = BAR(kv_free[0]);
      if (p.debug_stall) {
        const uint64_t s0 = ptx::globaltimer();
        while (!ctl->abort && ptx::globaltimer() - s0 < 4ull * p.wait_limit_ns) {
        }
        if (!ctl->abort) wt.give_up();
        ok = false;
      }
      while (ok) {
        if (!wt.wait(bar_kv + (u & 1) * 8, (u >> 1) & 1)) break;
        const uint32_t f = ctl->ring[u & 3];
        ptx::tc_fence_after();
        bool need_q = (f & kItemFirst) != 0u;
        auto pv = [&](int g) -> bool {
          if ((prev & (kFirst0 << g)) && (prev & kItemAfterFirst) &&
              !wt.wait(BAR(o_free[g]), (prev & kItemOdd) ? 0u : 1u))
            return false;
          if (!wt.wait(BAR(p_full[g]), pc[g] & 1)) return false;
          ++pc[g];
          ptx::tc_fence_after();
          const uint32_t p_tmem = tmem + C::S_COL + g * BN;
          const uint32_t o_tmem = tmem + C::O_COL + g * D;
          const uint64_t vd = v_desc0 + uint64_t((((u - 1) & 1) * C::KV_BYTES) >> 4);
          const bool fresh = (prev & (kFirst0 << g)) != 0u;
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            ptx::mma_ts(o_tmem, p_tmem + kk * 8, vd + uint64_t(kk * 128), C::IDESC_PV, (fresh && kk == 0) ? 0u : 1u);
          if (prev & (kLast0 << g)) ptx::mma_commit(BAR(pv_done[g]));
          return true;
        };
        auto qk = [&](int g) -> bool {
          if (need_q) {
            if (!wt.wait(BAR(q_full), (f & kItemOdd) ? 1u : 0u)) return false;
            ptx::tc_fence_after();
            need_q = false;
          }
          const uint64_t qd = q_desc0 + uint64_t((((f & kSpanAlt) ? 0 : g) * C::Q_BYTES) >> 4);
          const uint64_t kd = k_desc0 + uint64_t(((u & 1) * C::KV_BYTES) >> 4);
          const uint32_t s_tmem = tmem + C::S_COL + g * BN;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = uint64_t((kk >> 2) * (C::Q_CHUNK >> 4) + (kk & 3) * 2);
            const uint64_t offk = uint64_t((kk >> 2) * (C::KV_CHUNK >> 4) + (kk & 3) * 2);
            ptx::mma_ss(s_tmem, qd + off, kd + offk, C::IDESC_QK, kk > 0 ? 1u : 0u);
          }
          ptx::mma_commit(BAR(s_full[g]));
          return true;
        };
        if (prev & f & (kLive0 | kLive1)) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (ok && (prev & (kLive0 << g))) ok = pv(g);
            if (ok && (f & (kLive0 << g))) ok = qk(g);
          }
        } else {
          // The two tiles are for different groups (alternating ones above all): this tile's scores
          // need not wait for the other group's softmax.
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (ok && (f & (kLive0 << g))) ok = qk(g);
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (ok && (prev & (kLive0 << g))) ok = pv(g);
        }
        if (!ok || (f & kEnd)) break;
        ptx::mma_commit(bar_free + (u & 1) * 8);
        if (f & kItemLast) ptx::mma_commit(BAR(q_empty));
        prev = f;
        ++u;
      }
      ptx::mma_commit(BAR(drain));
      wt.wait_drain(BAR(drain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------- softmax warpgroups
    const int grp = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;       // TMEM lane
    const int row = F == 1 ? r : lane;       // row of the query tile
    const int col0 = F == 1 ? 0 : quarter * NC;  // this thread's first key column of a tile
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    const uint32_t gbar = 1 + grp;
    constexpr uint32_t kAll = 7;  // named barrier of both groups
    uint8_t* stage = smem + C::OFF_OST + (grp * 4 + quarter) * C::OST_WARP;
    float* kpos = reinterpret_cast<float*>(smem + C::OFF_OST + grp * 4 * C::OST_WARP);  // two tiles (bias)
    const uint32_t s_tmem = tmem + lane_base + C::S_COL + grp * BN;
    const uint32_t o_tmem = tmem + lane_base + C::O_COL + grp * D;
    const int r_tok = row / p.G, r_head = row - r_tok * p.G;
    // batch entry, token and head of this thread's row in the item
    auto row_of = [&](const SpanInfo* it, int& b, int& n, int& h) {
      b = it->b;
      n = it->t[grp].tok0 + r_tok;
      if (it->kind == 1) {
        b = n / p.Nq;
        n -= b * p.Nq;
      }
      h = it->hk * p.G + r_head;
    };
    uint32_t tg = 0, items = 0, pv_phase = 0;
    while (true) {
      const int slot = items & 1;
      bool ok = wt.wait(BAR(item_full[slot]), (items >> 1) & 1);
      const SpanInfo* it = &ctl->info[slot];  // released (item_empty) at the end of the item
      const SpanTile* mt = &it->t[grp];
      ++items;
      // (with F > 1 the groups meet in the epilogue, so they give up together)
      if (!ptx::named_bar_and(F > 1 ? kAll : gbar, F > 1 ? 256 : 128, ok) || it->kind < 0) break;
      const int n_live = mt->n_live;
      const bool valid = row < mt->rows;
      const bool warp_valid = F > 1 || quarter * 32 < mt->rows;  // the warp has a valid row
      int ks = 0, ke = 0;
      float slope = 0.f, qp = 0.f;
      if (valid) {
        int b, n, h;
        row_of(it, b, n, h);
        if (it->kind == 0) span_of(p, b, n, ks, ke);
        if (BIAS) {
          slope = __ldg(p.slopes + h) * 1.4426950408889634f;
          qp = p.q_pos ? __ldg(p.q_pos + b * p.q_pos_b + n) : float(p.Np + p.Nk - p.Nq + n);
        }
      }
      // no row of the warp has a slope too steep, or keys too far away, for the short way below
      bool gentle = true;
      if (BIAS)
        gentle = __all_sync(0xffffffffu, !valid || (fabsf(slope) * PC <= (CAP ? 30.f : 60.f) &&
                                                     fabsf(slope) * (fabsf(qp) + float(p.Np + p.Nk)) <= kSpanFarBias));
      float m_used = -INFINITY;  // exponent reference (lazy rescale), log2 units
      float l = 0.f;             // row sum relative to m_used
      // given position of key r of the group's tile idx
      auto key_pos = [&](int idx) -> float {
        const int entry = mt->q0 + idx * mt->step;
        const bool pre = entry < mt->n_pre;
        const int m = (pre ? it->v_first + entry : mt->j_first + entry - mt->n_pre) * BN + r;
        const float* at = pre ? p.p_pos : p.k_pos;
        if (!at || r >= BN || m >= (pre ? p.Np : p.Nk)) return __int_as_float(0x7fffffff);  // no key: NaN
        return __ldg(at + (pre ? 0 : it->b * p.k_pos_b) + m);
      };
      float kp_next = 0.f;
      if (BIAS && n_live > 0) kp_next = key_pos(0);
      for (int idx = 0; idx < n_live; ++idx) {
        const int entry = mt->q0 + idx * mt->step;
        const bool pre = entry < mt->n_pre;
        const int j0 = (pre ? it->v_first + entry : mt->j_first + entry - mt->n_pre) * BN;  // the tile's first key
        float* kp = kpos + (idx & 1) * (BN + 8);
        const bool given = BIAS && (pre ? p.p_pos : p.k_pos) != nullptr;
        if (given) {
          // thread r brings the position of key r (read a tile ahead), and each warp the first and last of its
          // keys; the buffer's last readers passed the barrier of the tile before
          span_publish<BN>(kp, kp_next, r);
          ptx::named_bar_sync(gbar, 128);
        }
        if (BIAS && idx + 1 < n_live) kp_next = key_pos(idx + 1);
        bool masked = false;   // some row of the query tile does not see all keys of this tile
        bool unclean = false;  // some row of the item that has this tile does not see all keys that it holds
        if (pre) {
          masked = p.Np - j0 < BN;
        } else if (j0 < mt->quiet_lo || j0 + BN > mt->quiet_hi) {
          const SpanTile& ot = it->t[grp ^ 1];  // (alternating groups: the same query tile)
          const int j = j0 / BN, oj = j - ot.j_first;
          masked = mt->full_lo > j0 || mt->full_hi < j0 + BN;
          unclean = span_cuts<BN>(p, *mt, j) ||
                    (F == 1 && oj >= 0 && oj < ot.n_live - ot.n_pre && span_cuts<BN>(p, ot, j));
        }
        wt.wait(BAR(s_full[grp]), tg & 1);
        ++tg;
        __syncwarp();
        ptx::tc_fence_after();
        if (warp_valid) {
          // Key x of the tile (default positions) is at distance |base + x|; where all rows of the warp have the
          // tile on one side, the bias is linear in x: sg * (base + x).
          const float base = BIAS ? float(j0 + col0 + (pre ? 0 : p.Np)) - qp : 0.f;
          const float sg = base < 0.f ? slope : -slope;
          bool fast = !masked && !given;
          if (BIAS)
            fast = fast && gentle && __all_sync(0xffffffffu, !valid || base >= 0.f || base <= 1.f - NC);
          float loc = -INFINITY;  // the tile's row maximum, or a reference near it (log2 units)
          float v[MOD == 0 ? NC / PC : 2][PC];
          if (fast) {
            // The exponents of a row need a reference near its maximum, not the maximum: P has the same
            // relative precision at every scale. With a cap or a bias it is at most 2 * 24 + 30 above (the
            // largest |score| taken for the score under a cap, the bias's spread over 32 columns; 60
            // without a cap), and 2^-78 is far from the end of the range. So it comes from the raw scores, and
            // the cap and the bias are packed products inside the exponent. The scores are read from
            // TMEM twice then, 32 at a time: a whole row in registers leaves too few of them to keep these
            // longer chains apart. Without cap and bias the row is read once and stays in registers.
            if constexpr (MOD == 0) {
#pragma unroll
              for (int c = 0; c < NC / PC; ++c) span_load<PC>(s_tmem + col0 + c * PC, v[c]);
              ptx::tmem_wait_ld();
              float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < NC / PC; ++c) span_max<PC>(v[c], m);
              loc = span_max4(m) * p.scale_log2;
            } else {
              float top = -INFINITY;
              span_load<PC>(s_tmem + col0, v[0]);
#pragma unroll
              for (int c = 0; c < NC / PC; ++c) {
                ptx::tmem_wait_ld();
                if (c + 1 < NC / PC) span_load<PC>(s_tmem + col0 + (c + 1) * PC, v[(c + 1) & 1]);
                float m[4];
                if constexpr (CAP) {
#pragma unroll
                  for (int x = 0; x < 4; ++x) m[x] = 0.f;
#pragma unroll
                  for (int x = 0; x < PC; x += 2) m[(x >> 1) & 3] = abs_max3(m[(x >> 1) & 3], v[c & 1][x], v[c & 1][x + 1]);
                } else {
#pragma unroll
                  for (int x = 0; x < 4; ++x) m[x] = -INFINITY;
                  span_max<PC>(v[c & 1], m);
                }
                const float here = span_max4(m);
                top = fmaxf(top, here);
                // (the cap only lowers a score; the bias is largest at one end of the chunk)
                if (BIAS)
                  loc = fmaxf(loc, fmaf(here, p.scale_log2, fmaxf(sg * (base + float(PC * c)), sg * (base + float(PC * c + PC - 1)))));
              }
              if (CAP) fast = !__any_sync(0xffffffffu, valid && !(top <= p.cap_near));
              if (!BIAS) loc = top * p.scale_log2;
            }
          }
          if (fast) {
            // lazy rescale of the accumulator, as in lite_attn_kernel
            const bool need = loc > m_used + kRescaleLog2;
            float alpha = 1.f;
            if (need) {
              alpha = ptx::ex2(m_used - loc);
              m_used = loc;
              l *= alpha;
            }
            // a row that has seen no key yet keeps m_used = -inf; its exponents are -inf - 0
            const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // bias minus reference of columns 2y, 2y + 1 of each eight, stepped from one eight to the next (at
            // most 16 sums: off by 2^-20 of an exponent that matters)
            float2 w[4];
            const float c0 = fmaf(sg, base, neg_m);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = BIAS ? make_float2(fmaf(sg, float(2 * y), c0), fmaf(sg, float(2 * y + 1), c0))
                          : make_float2(neg_m, neg_m);
            const float2 sg8 = make_float2(8.f * sg, 8.f * sg);
            if constexpr (MOD != 0) span_load<PC>(s_tmem + col0, v[0]);
#pragma unroll
            for (int c = 0; c < NC / PC; ++c) {
              if constexpr (MOD != 0) {
                ptx::tmem_wait_ld();
                if (c + 1 < NC / PC) span_load<PC>(s_tmem + col0 + (c + 1) * PC, v[(c + 1) & 1]);
              }
              const float(&vc)[PC] = v[MOD == 0 ? c : (c & 1)];
              span_put<PC>(s_tmem + col0 / 2 + c * (PC / 2), acc, [&](int x) {
                const float2 a = make_float2(vc[x], vc[x + 1]);
                float2& wx = w[(x >> 1) & 3];
                const float2 add = wx;
                if (BIAS) wx = __fadd2_rn(wx, sg8);
                if constexpr (CAP) {
                  // cap tanh(s scale / cap) as an odd polynomial: two exponential-unit operations a score
                  // more would triple the work of the unit that bounds the kernel
                  const float2 y = __fmul2_rn(a, a);
                  float2 t = __ffma2_rn(make_float2(p.cap_b[4], p.cap_b[4]), y, make_float2(p.cap_b[3], p.cap_b[3]));
                  t = __ffma2_rn(t, y, make_float2(p.cap_b[2], p.cap_b[2]));
                  t = __ffma2_rn(t, y, make_float2(p.cap_b[1], p.cap_b[1]));
                  t = __ffma2_rn(t, y, make_float2(p.cap_b[0], p.cap_b[0]));
                  return __ffma2_rn(a, t, add);
                } else {
                  return __ffma2_rn(a, sc2, add);
                }
              });
            }
            if constexpr (F > 1) span_zero<NC>(s_tmem, quarter);
            if (__any_sync(0xffffffffu, need) && idx >= 1) span_rescale<D>(o_tmem, alpha);
            ptx::tmem_wait_st();
            const float2 acc2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
            l += acc2.x + acc2.y;
          } else {
            // columns [lo, hi) of the tile are keys that this row sees
            const float2 ml = span_tile_in_full<D, NC, MOD, F>(
                p, s_tmem, o_tmem, quarter, (pre || !masked) ? 0 : ks - j0 - col0,
                !masked ? NC : (pre ? p.Np : ke) - j0 - col0, base, slope, qp, given ? kp + col0 : nullptr,
                make_float2(m_used, l), idx >= 1);
            m_used = ml.x;
            l = ml.y;
          }
        }
        if (unclean) {
          // Rows that do not see all keys of this tile have P = 0 there, but 0 times an infinity or NaN is
          // NaN: such values (whatever lies behind a sequence's end, say) are taken out of V before the
          // product, and rows that do see them get them back in the epilogue.
          span_clean_tile<C, BN>(ctl, smem, wt, slot, quarter * 32 + lane, j0 / BN, entry);
          __syncwarp();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(BAR(p_full[grp]));
      }
      // ----- epilogue
      if (BIAS && F == 1) ptx::named_bar_sync(gbar, 128);  // the position buffer becomes the staging area
      if (n_live > 0) {
        wt.wait(BAR(pv_done[grp]), pv_phase & 1);
        ++pv_phase;
        __syncwarp();
        ptx::tc_fence_after();
        if (warp_valid && *static_cast<volatile const int*>(&it->n_bad) > 0) {
          int b, n, h;
          row_of(it, b, n, h);
          span_repair<D, BN, NC>(p, *it, grp, o_tmem, valid, ks, ke, b, col0);
        }
      }
      // a row that saw no key: o = 0, lse = -inf (l is 0 then; a NaN score leaves its mark in l)
      const bool empty = l == 0.f;
      if constexpr (F > 1) {
        // The row's eight partial results (four quarters, two groups) are joined here, 32 columns at a time
        // through the staging area: thread x of the 256 takes row x / 8 and four columns of each 32.
        float* ml = reinterpret_cast<float*>(smem + C::OFF_OST);
        const int src = grp * 4 + quarter, x256 = grp * 128 + quarter * 32 + lane;
        const int orow = x256 >> 3, quad = x256 & 7;
        ptx::named_bar_sync(kAll, 256);
        *reinterpret_cast<float2*>(ml + (src * 32 + lane) * 2) = make_float2(m_used, l);
        ptx::named_bar_sync(kAll, 256);
        float mm = -INFINITY, tot = 0.f, w[8];
        uint32_t seen = 0u;  // the partial results that saw a key (the others' O may be anything)
#pragma unroll
        for (int y = 0; y < 8; ++y) mm = fmaxf(mm, ml[(y * 32 + orow) * 2]);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float2 e = *reinterpret_cast<const float2*>(ml + (y * 32 + orow) * 2);
          w[y] = e.y == 0.f ? 0.f : (mm == -INFINITY ? 1.f : ptx::ex2(e.x - mm));
          if (e.y != 0.f) {
            tot = fmaf(w[y], e.y, tot);
            seen |= 1u << y;
          }
        }
        ptx::named_bar_sync(kAll, 256);
        const bool o_valid = orow < mt->rows;
        const float inv = p.part ? 1.f : (tot == 0.f ? 0.f : 1.f / tot);
        int b = it->b, n = mt->tok0 + orow / p.G;
        if (it->kind == 1) {
          b = n / p.Nq;
          n -= b * p.Nq;
        }
        const int h = it->hk * p.G + orow % p.G;
        float* part = p.part + (it->kind == 1 ? p.pre : p.own).part0 + it->slot * span_part_floats(D, PR);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t rr[32];
          ptx::tmem_ld32(o_tmem + c * 32, rr);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                make_uint4(rr[4 * x], rr[4 * x + 1], rr[4 * x + 2], rr[4 * x + 3]);
          ptx::named_bar_sync(kAll, 256);
          float4 acc4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            if (!(seen & (1u << y))) continue;
            const float4 e = *reinterpret_cast<const float4*>(smem + C::OFF_OST + y * C::OST_WARP + orow * 128 +
                                                              ((quad ^ (orow & 7)) << 4));
            acc4.x = fmaf(w[y], e.x, acc4.x);
            acc4.y = fmaf(w[y], e.y, acc4.y);
            acc4.z = fmaf(w[y], e.z, acc4.z);
            acc4.w = fmaf(w[y], e.w, acc4.w);
          }
          if (o_valid) {
            if (p.part) {
              *reinterpret_cast<float4*>(part + orow * D + c * 32 + quad * 4) = acc4;
            } else {
              const __nv_bfloat162 a = __floats2bfloat162_rn(acc4.x * inv, acc4.y * inv),
                                   z = __floats2bfloat162_rn(acc4.z * inv, acc4.w * inv);
              *reinterpret_cast<uint2*>(p.o + ((static_cast<long long>(b) * p.Nq + n) * p.H + h) * D + c * 32 + quad * 4) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&z));
            }
          }
          ptx::named_bar_sync(kAll, 256);
        }
        ptx::tc_fence_before();
        if (it->t[0].n_live + it->t[1].n_live > 0) ptx::mbar_arrive(BAR(o_free[grp]));
        if (o_valid && quad == 0) {
          if (p.part) {
            part[PR * D + orow] = mm;
            part[PR * D + PR + orow] = tot;
          } else if (p.lse) {
            p.lse[(size_t(b) * p.H + h) * p.Nq + n] =
                tot == 0.f ? -INFINITY : (mm + __log2f(tot)) * 0.6931471805599453f;
          }
        }
      } else if (p.part) {
        float* part = p.part + (it->kind == 1 ? p.pre : p.own).part0 + (it->slot + grp) * span_part_floats(D, PR);
        if (warp_valid) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t rr[32];
            ptx::tmem_ld32(o_tmem + c * 32, rr);
            ptx::tmem_wait_ld();
              float4* dst = reinterpret_cast<float4*>(part + r * D + c * 32);
            // (a part without keys is not read: its row sum says so)
            if (valid && !empty)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[x] = make_float4(__uint_as_float(rr[4 * x]), __uint_as_float(rr[4 * x + 1]),
                                     __uint_as_float(rr[4 * x + 2]), __uint_as_float(rr[4 * x + 3]));
          }
          if (valid) {
            part[PR * D + r] = m_used;
            part[PR * D + PR + r] = l;
          }
        }
        ptx::tc_fence_before();
        if (it->t[0].n_live + it->t[1].n_live > 0) ptx::mbar_arrive(BAR(o_free[grp]));
      } else {
        // Rows go out through the warp's staging area, 64 columns of its 32 rows at a time, so that
        // its lanes write 128-byte pieces (a tile's rows may belong to several tokens, heads and batch
        // entries, so there is no box to store).
        const float inv_l = empty ? 0.f : 1.f / l;
        int b, n, h;
        row_of(it, b, n, h);
        const long long o_row = (static_cast<long long>(b) * p.Nq + n) * p.H + h;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          if (!warp_valid) break;
          __syncwarp();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t rr[32];
            ptx::tmem_ld32(o_tmem + c * 64 + half * 32, rr);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float a = __uint_as_float(rr[8 * x + 2 * y]) * inv_l;
                const float z = __uint_as_float(rr[8 * x + 2 * y + 1]) * inv_l;
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, z);
                w[y] = empty ? 0u : *reinterpret_cast<const uint32_t*>(&h2);
              }
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((half * 4 + x) ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int srow = i * 4 + (lane >> 3), x = lane & 7;
            const long long row = __shfl_sync(0xffffffffu, o_row, srow);
            if (quarter * 32 + srow < mt->rows)
              *reinterpret_cast<uint4*>(p.o + row * D + c * 64 + x * 8) =
                  *reinterpret_cast<const uint4*>(stage + srow * 128 + ((x ^ (srow & 7)) << 4));
          }
        }
        ptx::tc_fence_before();
        if (it->t[0].n_live + it->t[1].n_live > 0) ptx::mbar_arrive(BAR(o_free[grp]));
        if (valid && p.lse)
          p.lse[(size_t(b) * p.H + h) * p.Nq + n] =
              empty ? -INFINITY : (m_used + __log2f(l)) * 0.6931471805599453f;
        if (BIAS) ptx::named_bar_sync(gbar, 128);  // before the next item's positions overwrite the staging
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(BAR(item_empty[slot]));
    }
  }
#undef BAR

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the parts of every output row: M = max m_i, o = sum 2^(m_i - M) O_i / L, L = sum 2^(m_i - M) l_i.
// One group of D/4 lanes per row, which reads the maxima of its parts at once and then the parts four at
// a time. Bound by latency: the parts were written just before and are in L2.
template <int D>
__global__ void __launch_bounds__(256) lite_span_combine_kernel(const SpanParams p) {
  constexpr int L = D / 4;  // lanes of a row
  const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  if (row >= static_cast<long long>(p.B) * p.Nq * p.H) return;  // (whole groups of lanes)
  const int h = int(row % p.H);
  const long long bn = row / p.H;
  const int b = int(bn / p.Nq), n = int(bn - static_cast<long long>(b) * p.Nq);
  const int hk = h / p.G, gh = h - hk * p.G;
  const float* part[2];
  int count[2], at[2], rows[2];
  size_t step[2];  // from one part of the row to the next
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const SpanPass& ps = k ? p.own : p.pre;
    count[k] = 0;
    rows[k] = ps.rows;
    if (ps.pairs == 0) continue;
    const int tok = k ? n : int(bn), tile = tok / ps.TN;
    at[k] = (tok - tile * ps.TN) * p.G + gh;
    const int pair = ps.alt ? tile : tile >> 1, unit = k ? b * p.Hk + hk : hk;
    const size_t first = (size_t(unit) * ps.pairs + (ps.pairs - 1 - pair)) * ps.splits * ps.per_item;
    const size_t floats = span_part_floats(D, ps.rows);
    part[k] = p.part + ps.part0 + (first + (ps.alt ? 0 : tile & 1)) * floats;
    // alternating groups: every part of the item holds the row
    count[k] = ps.alt ? ps.splits * ps.per_item : ps.splits;
    step[k] = (ps.alt ? 1 : ps.per_item) * floats;
  }
  const int total = count[0] + count[1];
  const auto part_at = [&](int i) -> const float* {
    return i < count[0] ? part[0] + i * step[0] + at[0] * D : part[1] + (i - count[0]) * step[1] + at[1] * D;
  };
  // the scratch is written by the kernel before this one in the stream, which has ended but whose writes may not be seen yet
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float m = -INFINITY, tot = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const unsigned lanes = L == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);  // the row's lanes of the warp
  for (int base = 0; base < total; base += L) {
    // lane i brings maximum and sum of part base + i, then all lanes take the parts in order
    float mi = -INFINITY, li = 0.f;
    if (base + lane < total) {
      const int i = base + lane;
      const float* q = i < count[0] ? part[0] + i * step[0] + rows[0] * D + at[0]
                                    : part[1] + (i - count[0]) * step[1] + rows[1] * D + at[1];
      mi = q[0];
      li = q[i < count[0] ? rows[0] : rows[1]];
    }
    float top = mi;
#pragma unroll
    for (int x = L / 2; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, x));
    top = fmaxf(top, m);
    const float keep = m == top ? 1.f : exp2f(m - top);  // (m may be -inf: nothing is kept then)
    // a part that saw no key weighs nothing; one without a maximum but with a NaN sum passes it on
    const float wi = li == 0.f ? 0.f : (top == -INFINITY ? 1.f : exp2f(mi - top));
    m = top;
    acc.x *= keep;
    acc.y *= keep;
    acc.z *= keep;
    acc.w *= keep;
    tot *= keep;
    const int n = min(L, total - base);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float w = __shfl_sync(lanes, wi, i, L), lw = __shfl_sync(lanes, li, i, L);
      if (lw == 0.f) continue;
      const float4 x = *reinterpret_cast<const float4*>(part_at(base + i) + lane * 4);
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
      tot = fmaf(w, lw, tot);
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), z = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 out;
  out.x = *reinterpret_cast<const uint32_t*>(&a);
  out.y = *reinterpret_cast<const uint32_t*>(&z);
  *reinterpret_cast<uint2*>(p.o + row * D + lane * 4) = out;
  if (p.lse && lane == 0)
    p.lse[(size_t(b) * p.H + h) * p.Nq + n] = tot == 0.f ? -INFINITY : (m + log2f(tot)) * 0.6931471805599453f;
}

}  // namespace lite
