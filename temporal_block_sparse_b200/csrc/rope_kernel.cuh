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
// shared by all its heads. A thread's unit is 16 elements of one head, the 8-element chunks c and
// c + d/16: with halves these hold both elements of 8 pairs, with interleaved pairs they are
// complete by themselves, so one mapping serves both and the d/16 lanes of a head read whole
// 64- or 128-byte pieces. A block takes whole tokens (one, or several when a token has few heads).
// All of a thread's loads are issued before anything else, so that the position arithmetic and
// both barriers run under their latency.
//
// The angle is formed in 64 bits as turns, position * (f / 2 pi), and reduced to [-1/2, 1/2] before
// it becomes a 32-bit number: positions of a long stream reach 10^5 and more, where a 32-bit angle
// is off by 10^-2. Sums of squares are 32-bit: a head's in its lanes' shuffle tree, a row's over
// its heads in index order, the same on every run. The only rounding is the output's, to bf16.
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
  RopeTensor t[2];        // queries, keys (heads = 0: no keys)
  int tokens;             // B * N
  int N;
  int units;              // units of one token: (heads[0] + heads[1]) * d / 16
  int units_q;            // of which queries: heads[0] * d / 16
  int tpb;                // tokens per block
  int norm;               // 0 none, 1 over the head, 2 over the token's heads
  float eps;
  int n_axes;
  long long grid[kRopeMaxAxes];   // sizes of the token grid (pos == null), last axis fastest
  long long start;                // grid index of token 0
  const void* pos;                // [B or 1, axes, N] positions, or null
  int pos_is_int;
  long long pos_b, pos_a;         // strides of pos in elements
  double turns[kRopeMaxPairs];    // frequency / 2 pi of each pair
  uint8_t axis[kRopeMaxPairs];
};

// 8 consecutive elements as floats
struct Raw16 {
  uint4 v;
};
struct Raw32 {
  uint4 lo, hi;
};
template <typename T>
struct RopeIn;
template <>
struct RopeIn<__nv_bfloat16> {
  using Raw = Raw16;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) {
    return Raw{__ldcs(reinterpret_cast<const uint4*>(p))};
  }
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r.v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = __bfloat1622float2(h[e]);
      f[2 * e] = a.x;
      f[2 * e + 1] = a.y;
    }
  }
};
template <>
struct RopeIn<__half> {
  using Raw = Raw16;
  static __device__ __forceinline__ Raw load(const __half* p) {
    return Raw{__ldcs(reinterpret_cast<const uint4*>(p))};
  }
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&r.v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = __half22float2(h[e]);
      f[2 * e] = a.x;
      f[2 * e + 1] = a.y;
    }
  }
};
template <>
struct RopeIn<float> {
  using Raw = Raw32;
  static __device__ __forceinline__ Raw load(const float* p) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    return Raw{__ldcs(q), __ldcs(q + 1)};
  }
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[8]) {
    const float* a = reinterpret_cast<const float*>(&r.lo);
    const float* b = reinterpret_cast<const float*>(&r.hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  }
};

__device__ __forceinline__ uint4 rope_pack(const float (&f)[8]) {
  uint4 r;
  uint32_t* o = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    o[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}

// position of token (b, n) on axis a
__device__ __forceinline__ double rope_position(const RopeParams& p, int b, int n, int a) {
  if (p.pos) {
    const long long at = b * p.pos_b + a * p.pos_a + n;
    return p.pos_is_int ? double(static_cast<const int*>(p.pos)[at]) : double(static_cast<const float*>(p.pos)[at]);
  }
  unsigned long long i = static_cast<unsigned long long>(p.start) + n;
  unsigned long long at = 0;
  // the grid index holds below 2^32 for all but very long streams: then 32-bit divisions do
  for (int x = p.n_axes - 1; x >= a; --x) {
    const unsigned long long g = static_cast<unsigned long long>(p.grid[x]);
    unsigned long long next;
    if ((i | g) >> 32)
      next = i / g;
    else
      next = uint32_t(i) / uint32_t(g);
    at = i - next * g;
    i = next;
  }
  return double(at);
}

// Shared memory: [tpb][D/2] (cos, sin) | [tpb][heads] sums of squares | [tpb][2] scale of the row
template <typename T, int D, bool HALVES, int U>
__global__ void lite_rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float rope_smem[];
  constexpr int C = D / 16;  // units (lanes) per head
  const int heads = p.t[0].heads + p.t[1].heads;
  float2* cs = reinterpret_cast<float2*>(rope_smem);
  float* hsum = rope_smem + p.tpb * D;
  float* rscale = hsum + p.tpb * heads;
  const int first = int(blockIdx.x) * p.tpb;
  const int n_tok = min(p.tpb, p.tokens - first);
  const int total = n_tok * p.units;
  using In = RopeIn<T>;

  typename In::Raw lo[U], hi[U];
  int tok[U], head[U], chunk[U], which[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int flat = u * blockDim.x + threadIdx.x;
    tok[u] = -1;
    if (flat < total) {
      const int tk = flat / p.units;
      int rem = flat - tk * p.units;
      const int w = rem >= p.units_q;
      rem -= w ? p.units_q : 0;
      tok[u] = tk;
      which[u] = w;
      head[u] = rem / C;
      chunk[u] = rem % C;
      const int b = (first + tk) / p.N, n = first + tk - b * p.N;
      const RopeTensor& x = p.t[w];
      const T* src = static_cast<const T*>(x.x) + b * x.xs[0] + n * x.xs[1] + head[u] * x.xs[2] + chunk[u] * 8;
      lo[u] = In::load(src);
      hi[u] = In::load(src + D / 2);
    }
  }

  for (int i = threadIdx.x; i < n_tok * (D / 2); i += blockDim.x) {
    const int tk = i / (D / 2), pr = i % (D / 2);
    const int b = (first + tk) / p.N, n = first + tk - b * p.N;
    const double turn = rope_position(p, b, n, p.axis[pr]) * p.turns[pr];
    float s, c;
    sincospif(2.0f * float(turn - rint(turn)), &s, &c);
    cs[i] = make_float2(c, s);
  }

  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) scale[u] = 1.f;
  if (p.norm) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float ss = 0.f;
      if (tok[u] >= 0) {
        float a[8], b[8];
        In::get(lo[u], a);
        In::get(hi[u], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
      }
#pragma unroll
      for (int m = C / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      if (p.norm == 1) {
        scale[u] = rsqrtf(ss * (1.0f / D) + p.eps);
      } else if (tok[u] >= 0 && chunk[u] == 0) {
        hsum[tok[u] * heads + (which[u] ? p.t[0].heads : 0) + head[u]] = ss;
      }
    }
  }
  __syncthreads();
  if (p.norm == 2) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int i = warp; i < n_tok * 2; i += warps) {
      const int w = i & 1, h0 = w ? p.t[0].heads : 0, nh = p.t[w].heads;
      const float* src = hsum + (i >> 1) * heads + h0;
      float ss = 0.f;
      for (int h = lane; h < nh; h += 32) ss += src[h];
#pragma unroll
      for (int m = 16; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      if (lane == 0 && nh > 0) rscale[i] = rsqrtf(ss / (float(nh) * D) + p.eps);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (tok[u] >= 0) scale[u] = rscale[tok[u] * 2 + which[u]];
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (tok[u] < 0) continue;
    const RopeTensor& x = p.t[which[u]];
    float a[8], b[8];
    In::get(lo[u], a);
    In::get(hi[u], b);
    if (p.norm) {
      const float* w = x.w + (p.norm == 2 ? head[u] * D : 0) + chunk[u] * 8;
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(w)), w1 = __ldg(reinterpret_cast<const float4*>(w) + 1);
      const float4 w2 = __ldg(reinterpret_cast<const float4*>(w + D / 2)),
                   w3 = __ldg(reinterpret_cast<const float4*>(w + D / 2) + 1);
      const float wa[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      const float wb[8] = {w2.x, w2.y, w2.z, w2.w, w3.x, w3.y, w3.z, w3.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] *= scale[u] * wa[e];
        b[e] *= scale[u] * wb[e];
      }
    }
    const float2* t = cs + tok[u] * (D / 2);
    float ya[8], yb[8];
    if (HALVES) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 r = t[chunk[u] * 8 + e];
        ya[e] = a[e] * r.x - b[e] * r.y;
        yb[e] = a[e] * r.y + b[e] * r.x;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 r = t[chunk[u] * 4 + e], s = t[D / 4 + chunk[u] * 4 + e];
        ya[2 * e] = a[2 * e] * r.x - a[2 * e + 1] * r.y;
        ya[2 * e + 1] = a[2 * e] * r.y + a[2 * e + 1] * r.x;
        yb[2 * e] = b[2 * e] * s.x - b[2 * e + 1] * s.y;
        yb[2 * e + 1] = b[2 * e] * s.y + b[2 * e + 1] * s.x;
      }
    }
    const int b0 = (first + tok[u]) / p.N, n = first + tok[u] - b0 * p.N;
    __nv_bfloat16* dst = x.y + b0 * x.ys[0] + n * x.ys[1] + head[u] * x.ys[2] + chunk[u] * 8;
    *reinterpret_cast<uint4*>(dst) = rope_pack(ya);
    *reinterpret_cast<uint4*>(dst + D / 2) = rope_pack(yb);
  }
}

}  // namespace lite
