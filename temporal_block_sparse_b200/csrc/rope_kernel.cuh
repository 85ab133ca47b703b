// rope_kernel.cuh -- RMS norm of queries and keys fused with rotary positions on several axes.
//
// For one token n and one head of d elements:
//   x <- x * rsqrt(mean(x^2) + eps) * w        (mean over the head, or over all heads of the token;
//                                               optional)
//   pair p = 0 .. d/2-1 belongs to axis a(p) (frame, row, column, ...) and has frequency f(p):
//   phi = position_a(p)(n) * f(p),  (x0, x1) <- (x0 cos phi - x1 sin phi, x0 sin phi + x1 cos phi)
// with (x0, x1) = elements (2p, 2p+1) (interleaved) or (p, p + d/2) (halves).
//
// HBM-bound: every element is read once and written once; the weights and the angles of a token are
// shared by all its heads. A thread's unit is 16 elements of one head in 16-byte pieces (two of bf16 or fp16,
// four of fp32): piece j of lane c holds elements j * d / pieces + c * (elements of a piece) and on, so the
// d/16 lanes of a head read and write whole 32-byte sectors side by side, interleaved pairs lie
// within a piece, and with halves piece j pairs with piece j + pieces / 2. Blocks are persistent, each
// for queries or for keys, and take whole tokens (one, or several when a token has few heads); a
// thread keeps its place in the token, so that little index arithmetic is left in the loop. The data
// of the next tokens come in by asynchronous copies (each thread copies what it will read itself, so they
// need no barrier), and their angles are computed beside the present work: one barrier per step is
// left (none, but for new angles, without a row norm), and the loads never stop.
//
// Measured (B200, 6.55 TB/s copy): 720p layer, 75600 tokens x 2 x 40 heads, d = 128, bf16, row norm: 565-613 us
// for 3.10 GB (0.77-0.84 of the copy); 480p, d = 64, fp32 in, head norm: 155-170 us for 1.01 GB (0.91-0.99).
// Fewer blocks with more registers (128) beat more blocks (64 registers: 15% slower), fewer stages more
// (see RopeCfg). The row norm's barrier keeps the first from the second's rate.
//
// Angles are formed in 64 bits and reduced to half a turn either way before they become 32-bit
// numbers: positions of a long stream reach 10^5 and more, where a 32-bit angle is off by 10^-2. For whole
// positions the turns of a pair are a 64-bit fraction, position * frequency / 2 pi modulo 1 being one
// integer product that wraps; other positions take a product of doubles. cos and sin of the reduced
// angle come from the special function unit (off by at most 2^-20.5, an output's rounding is
// 2^-9 and more). Sums of squares are 32-bit, in a fixed order. The only rounding is the output's, to bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace lite {

constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxPairs = 64;

struct RopeTensor {
  const void* x;          // [B, N, heads, d], any 16-byte aligned strides
  __nv_bfloat16* y;       // [B, N, heads, d]
  const float* w;         // [d] or [heads * d] or null
  long long xs[3];        // strides in elements: batch, token, head
  long long ys[3];
  int heads;
};

struct RopeParams {
  RopeTensor t[2];        // queries, keys
  int q_blocks;           // blocks 0 .. q_blocks-1 take queries, the others keys
  int halves;             // pairs (p, p + d/2) instead of (2p, 2p + 1)
  int tokens;             // B * N
  int N;
  uint64_t n_magic;       // floor(2^63 / N) + 1: t / N = (2 t n_magic) >> 64 for t < 2^31
  float eps;
  int n_axes;
  long long grid[kRopeMaxAxes];   // sizes of the token grid (pos == null), last axis fastest
  long long start;                // grid index of token 0
  const void* pos;                // [B or 1, axes, N] positions, or null
  int pos_is_int;
  int whole;              // positions are whole numbers: grid or int32
  long long pos_b, pos_a;         // strides of pos in elements
  double turns[kRopeMaxPairs];    // frequency / 2 pi of each pair; its fractional part times 2^64 as an
                                  // integer where positions are whole
  uint8_t axis[kRopeMaxPairs];
};

// The 16 bytes at `src` to shared memory, past the registers; complete after rope_copies_left().
__device__ __forceinline__ void rope_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void rope_copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's committed groups are under way
template <int N>
__device__ __forceinline__ void rope_copies_left() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// elements of one 16-byte piece, in pairs
__device__ __forceinline__ void rope_get(const uint4& v, const __nv_bfloat16*, float2* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = __bfloat1622float2(h[e]);
}
__device__ __forceinline__ void rope_get(const uint4& v, const __half*, float2* f) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = __half22float2(h[e]);
}
__device__ __forceinline__ void rope_get(const uint4& v, const float*, float2* f) {
  const float4 a = *reinterpret_cast<const float4*>(&v);
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
}

// N element pairs rounded to bf16 and stored (8 or 16 bytes)
template <int N>
__device__ __forceinline__ void rope_put(uint8_t* dst, const float2* f) {
  uint32_t o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[e].x, f[e].y);
    o[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if constexpr (N == 4)
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
}

// positions of token t on all axes: 64-bit integers (p.whole) or doubles
__device__ __forceinline__ void rope_positions(const RopeParams& p, int t, long long* at) {
  const int b = int(__umul64hi(uint64_t(t) << 1, p.n_magic)), n = t - b * p.N;
  if (p.pos) {
#pragma unroll
    for (int a = 0; a < kRopeMaxAxes; ++a) {
      if (a >= p.n_axes) break;
      const long long i = b * p.pos_b + a * p.pos_a + n;
      at[a] = p.pos_is_int ? static_cast<long long>(static_cast<const int*>(p.pos)[i])
                           : __double_as_longlong(double(static_cast<const float*>(p.pos)[i]));
    }
    return;
  }
  unsigned long long i = static_cast<unsigned long long>(p.start) + n;
#pragma unroll
  for (int a = kRopeMaxAxes - 1; a >= 0; --a) {
    if (a >= p.n_axes) continue;
    // the grid index is below 2^32 for all but very long streams: then a 32-bit division does
    const unsigned long long g = static_cast<unsigned long long>(p.grid[a]);
    const unsigned long long next = ((i | g) >> 32) ? i / g : uint32_t(i) / uint32_t(g);
    at[a] = static_cast<long long>(i - next * g);
    i = next;
  }
}

template <typename T, int U>
struct RopeCfg {
  static constexpr int E = 16 / sizeof(T);   // elements of a piece
  static constexpr int RC = 16 / E;          // pieces of a unit
  // Steps whose data are in shared memory or on their way. With 16-bit inputs three (a frame of 2 x 1560 tokens: 26.7
  // us, 28.7 with two; the 720p layer within 1%), with fp32 two (480p: 155-170 us, 178 with three).
  static constexpr int STAGES = sizeof(T) == 2 ? 3 : 2;
  static constexpr int STEP = U * RC * 16;   // bytes of a thread's step
};

// The sizes of a block's shared memory: [stages][U * RC][threads] 16-byte pieces | frequencies [D/2],
// axes [D/2] | two of each: positions [ahead][tpb][axes], (cos, sin) [ahead][tpb][D/2], sums of
// squares [max(tpb * heads, warps)].
struct RopeShape {
  int units;   // units of a token: heads * D / 16
  int tpb;     // tokens per block and step
  int ahead;   // steps whose angles are computed at once
  int threads;
  __host__ __device__ int slots() const { return ahead * tpb; }
  __host__ __device__ int sums(int heads) const { return (tpb * heads > 32 ? tpb * heads : 32); }
  __host__ __device__ size_t bytes(int data, int D, int heads) const {  // data: bytes of a thread's pieces
    return size_t(data) * threads + (D / 2) * 12 +
           2 * (size_t(slots()) * (kRopeMaxAxes * 8 + D * 4) + size_t(sums(heads)) * 4);
  }
};

// NORM: 0 none, 1 over the head, 2 over the token's heads. ONE: one token a step.
template <typename T, int D, int U, int NORM, bool ONE>
__global__ void __maxnreg__(128) lite_rope_kernel(const __grid_constant__ RopeParams p, const RopeShape sq,
                                                         const RopeShape sk) {
  extern __shared__ __align__(16) uint8_t rope_smem[];
  constexpr int C = D / 16;  // units (lanes) per head
  using R = RopeCfg<T, U>;
  const bool keys = int(blockIdx.x) >= p.q_blocks;
  const RopeShape sh = keys ? sk : sq;
  const RopeTensor& x = p.t[keys];
  const int block = keys ? int(blockIdx.x) - p.q_blocks : int(blockIdx.x);
  const int n_blocks = keys ? int(gridDim.x) - p.q_blocks : p.q_blocks;
  const int tpb = ONE ? 1 : sh.tpb, stride = n_blocks * tpb, heads = x.heads;
  const int tid = threadIdx.x, threads = sh.threads, lane = tid & 31, warp = tid >> 5;
  if (tid >= threads) return;  // (the other tensor's blocks are larger); barriers count `threads`
  uint8_t* const pieces = rope_smem + tid * 16;
  double* const turns = reinterpret_cast<double*>(rope_smem + R::STAGES * R::STEP * threads);
  int* const axis = reinterpret_cast<int*>(turns + D / 2);
  long long* const places = reinterpret_cast<long long*>(axis + D / 2);  // [2][slots][axes]
  const int slots = sh.slots();
  float* const tables = reinterpret_cast<float*>(places + 2 * slots * kRopeMaxAxes);
  float* const sums = tables + 2 * slots * D;
  const auto barrier = [&]() { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); };

  // This thread's units: token slot, head, chunk (the same for all of them where a step is one token).
  int slot[U], head[U];
  const int chunk = tid % C;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int flat = u * threads + tid;
    slot[u] = flat / sh.units;  // tpb (ONE: not 0) for a thread without a unit
    head[u] = (flat - slot[u] * sh.units) / C;
  }
  auto mine = [&](int u, int first) { return slot[u] < tpb && (ONE || first + slot[u] < p.tokens); };
  // Where unit 0 of this thread's tokens starts: a cursor steps through the tokens of the block (ONE), an
  // address is made anew only where a batch entry ends.
  struct Cursor {
    const uint8_t* at;
    int n;  // token within its batch entry
  };
  auto place = [&](int t, const void* base, const long long* st, int h, int size) -> Cursor {
    const int b = int(__umul64hi(uint64_t(t) << 1, p.n_magic)), n = t - b * p.N;
    return Cursor{static_cast<const uint8_t*>(base) + (b * st[0] + n * st[1] + h * st[2] + chunk * R::E) * size, n};
  };
  auto advance = [&](Cursor& c, int t, long long step, const void* base, const long long* st, int size) {
    c.n += stride;
    c.at += step;
    if (c.n >= p.N) c = place(t, base, st, head[0], size);
  };
  const long long in_step = stride * x.xs[1] * int(sizeof(T)), out_step = stride * x.ys[1] * 2;
  // from one unit of the thread to its next one
  const long long in_unit = (threads / C) * x.xs[2] * int(sizeof(T)), out_unit = (threads / C) * x.ys[2] * 2;
  Cursor src_at = {nullptr, 0}, dst_at = {nullptr, 0};
  auto load = [&](long long first, int stage) {
    if (first < p.tokens) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!mine(u, int(first))) continue;
        const uint8_t* src = ONE ? src_at.at + u * in_unit : place(int(first) + slot[u], x.x, x.xs, head[u], sizeof(T)).at;
        uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(pieces)) + (stage * U + u) * R::RC * 16 * threads;
#pragma unroll
        for (int c = 0; c < R::RC; ++c) {
          rope_copy16(dst, src + c * (D / R::RC) * sizeof(T));
          dst += 16 * threads;
        }
      }
      if (ONE && first + stride < p.tokens)
        advance(src_at, int(first) + stride, in_step, x.x, x.xs, int(sizeof(T)));
    }
    rope_copies_commit();
  };
  // positions and angles of the steps from token `first` on, into table `which`
  auto fill_places = [&](long long first, int which) {
    for (int i = tid; i < slots; i += threads) {
      const long long t = first + static_cast<long long>(i / tpb) * stride + i % tpb;
      if (t < p.tokens) rope_positions(p, int(t), places + (which * slots + i) * kRopeMaxAxes);
    }
  };
  auto fill_angles = [&](int which) {
    for (int i = tid; i < slots * (D / 2); i += threads) {
      const int s = which * slots + i / (D / 2), pr = i % (D / 2);
      const long long at = places[s * kRopeMaxAxes + axis[pr]];
      float half_turns;  // [-1, 1]
      if (p.whole) {
        const unsigned long long f = static_cast<unsigned long long>(at) * static_cast<unsigned long long>(__double_as_longlong(turns[pr]));
        half_turns = float(int(f >> 32)) * 4.656612873077393e-10f;  // 2^-31
      } else {
        const double turn = __longlong_as_double(at) * turns[pr];
        half_turns = 2.0f * float(turn - rint(turn));
      }
      const float phi = half_turns * 3.14159265358979f;
      // entries of two (cos, sin) pairs, in the order in which the lanes of a head read them: entry e of
      // piece j, lane c at (j * entries of a piece + e) * C + c
      constexpr int PIECE = D / R::RC;
      const int el = p.halves ? pr : 2 * pr, j = el / PIECE, rest = el % PIECE, c = rest / R::E;
      const int e = p.halves ? rest % R::E / 2 : rest % R::E / 4, per = p.halves ? R::E / 2 : R::E / 4;
      *reinterpret_cast<float2*>(tables + static_cast<size_t>(s) * D + ((j * per + e) * C + c) * 4 + (pr & 1) * 2) =
          make_float2(__cosf(phi), __sinf(phi));
    }
  };

  long long first = static_cast<long long>(block) * tpb;
  if (ONE && first < p.tokens) {
    src_at = place(int(first), x.x, x.xs, head[0], sizeof(T));
    dst_at = place(int(first), x.y, x.ys, head[0], 2);
  }
#pragma unroll
  for (int y = 0; y < R::STAGES - 1; ++y) load(first + static_cast<long long>(y) * stride, y);
  // weights of the thread's units: they stay in registers
  float4 w[NORM ? U : 1][4];
  if constexpr (NORM != 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (slot[u] >= tpb) continue;
      const float* src = x.w + (NORM == 2 ? head[u] * D : 0) + chunk * R::E;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[u][e] = __ldg(reinterpret_cast<const float4*>(src + 4 * e / R::E * (D / R::RC) + 4 * e % R::E));
    }
  }
  for (int i = tid; i < D / 2; i += threads) {
    turns[i] = p.turns[i];
    axis[i] = p.axis[i];
  }
  const long long table_span = static_cast<long long>(sh.ahead) * stride;
  fill_places(first, 0);
  fill_places(first + table_span, 1);
  barrier();
  fill_angles(0);
  barrier();

  int stage = 0, in_table = 0, table = 0;  // place of the step in its angle table, and which of the two
  for (int step = 0; first < p.tokens; first += stride, ++step) {
    // the stage loaded into was read by this thread in the step before
    load(first + static_cast<long long>(R::STAGES - 1) * stride, stage == 0 ? R::STAGES - 1 : stage - 1);
    rope_copies_left<R::STAGES - 1>();
    float* hsum = sums + (step & 1) * sh.sums(heads);
    uint4 raw[U][R::RC];
    float ss[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* src = pieces + (stage * U + u) * R::RC * 16 * threads;
#pragma unroll
      for (int c = 0; c < R::RC; ++c) raw[u][c] = *reinterpret_cast<const uint4*>(src + c * 16 * threads);
    }
    constexpr int P2 = R::E / 2;  // element pairs of a piece
    auto get = [&](int u, float2 (&v)[8]) {
#pragma unroll
      for (int c = 0; c < R::RC; ++c) rope_get(raw[u][c], static_cast<const T*>(nullptr), v + c * P2);
    };
    if constexpr (NORM != 0) {
      float all = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float2 q = make_float2(0.f, 0.f);
        if (mine(u, int(first))) {
          float2 v[8];
          get(u, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) q = __ffma2_rn(v[e], v[e], q);
        }
        ss[u] = q.x + q.y;
        if (NORM == 1 || !ONE) {
#pragma unroll
          for (int m = C / 2; m; m >>= 1) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], m);
          if (NORM == 2 && slot[u] < tpb && chunk == 0) hsum[slot[u] * heads + head[u]] = ss[u];
        } else {
          all += ss[u];
        }
      }
      if (NORM == 2 && ONE) {
#pragma unroll
        for (int m = 16; m; m >>= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
        if (lane == 0) hsum[warp] = all;
      }
    }
    // new angles are seen from here on, and so are this step's sums
    if (NORM == 2 || in_table == 0) barrier();
    if (in_table == 0) {
      // The other table's last readers have passed the barrier, and so have the writers of its positions.
      // Positions for the table after it go where this table's were: read before the barrier.
      fill_angles(table ^ 1);
      fill_places(first + 2 * table_span, table);
    }
    float row = 0.f;
    if constexpr (NORM == 2 && ONE) {
      float sum = 0.f;
      for (int i = 0; i < threads / 32; ++i) sum += hsum[i];
      row = rsqrtf(sum / (float(heads) * D) + p.eps);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!mine(u, int(first))) continue;
      float2 v[8];
      get(u, v);
      if constexpr (NORM != 0) {
        float scale;
        if (NORM == 1) {
          scale = rsqrtf(ss[u] * (1.0f / D) + p.eps);
        } else if (ONE) {
          scale = row;
        } else {
          // a token with few heads: its sums in index order
          float sum = 0.f;
          for (int h = 0; h < heads; ++h) sum += hsum[slot[u] * heads + h];
          scale = rsqrtf(sum / (float(heads) * D) + p.eps);
        }
        const float2 s2 = make_float2(scale, scale);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __fmul2_rn(__fmul2_rn(v[2 * e], s2), make_float2(w[u][e].x, w[u][e].y));
          v[2 * e + 1] = __fmul2_rn(__fmul2_rn(v[2 * e + 1], s2), make_float2(w[u][e].z, w[u][e].w));
        }
      }
      const float4* cs = reinterpret_cast<const float4*>(
                             tables + static_cast<size_t>(table * slots + in_table * tpb + slot[u]) * D) + chunk;
      float2 y[8];
      if (p.halves) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // e / P2: piece, e % P2: entry
          const float4 r = cs[e * C];
          const float2 a = v[e], b = v[e + 4];
          y[e] = make_float2(a.x * r.x - b.x * r.y, a.y * r.z - b.y * r.w);
          y[e + 4] = make_float2(a.x * r.y + b.x * r.x, a.y * r.w + b.y * r.z);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 r = cs[e * C];
          const float2 a = v[2 * e], b = v[2 * e + 1];
          y[2 * e] = make_float2(a.x * r.x - a.y * r.y, a.x * r.y + a.y * r.x);
          y[2 * e + 1] = make_float2(b.x * r.z - b.y * r.w, b.x * r.w + b.y * r.z);
        }
      }
      uint8_t* dst = const_cast<uint8_t*>(ONE ? dst_at.at + u * out_unit
                                              : place(int(first) + slot[u], x.y, x.ys, head[u], 2).at);
#pragma unroll
      for (int c = 0; c < R::RC; ++c) rope_put<P2>(dst + c * (D / R::RC) * 2, y + c * P2);
    }
    if (ONE && first + stride < p.tokens) advance(dst_at, int(first) + stride, out_step, x.y, x.ys, 2);
    stage = stage + 1 == R::STAGES ? 0 : stage + 1;
    if (++in_table == sh.ahead) {
      in_table = 0;
      table ^= 1;
    }
  }
  rope_copies_left<0>();
}

}  // namespace lite
