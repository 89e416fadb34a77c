// Rotary positions, stand-alone: any positions, both channel layouts, part of the head, any
// table of frequencies, and the transpose of the rotation for the gradient.
//
// Channel pair i of a head vector at position m is turned by 2 pi m f_i, f_i in turns per
// token: (a, b) -> mscale (a cos - b sin, a sin + b cos); the gradient is the same with the
// opposite angle. Pair i is channels (2i, 2i+1) (interleaved) or (i, i + rot/2) (half);
// channels from `rot` on pass through.
//
// Bound by HBM: one read and one write of q and k. The angle is formed in fp64 and reduced to
// (-1/2, 1/2] turns before it is rounded, so that far positions lose nothing; sine and cosine
// are then fp32 (of the turn rounded to fp32: fp32 outputs are 5.1e-8 off, and 4.0e-8 with an fp64 angle). They are formed once per (token, pair) of a CTA's tile, in shared memory,
// and shared by all heads: fp64 work per token is rot/2 products. A thread keeps the (cos, sin) of its
// channels over the heads and has one row in flight; eight CTAs an SM then hide the latency better
// than more rows a thread (32768 tokens, 64 heads of 128 in bf16: 177 us, 6.1 TB/s, against 182 with
// two rows and 215 with four). Halves keep two runs and a (cos, sin) for each of their pairs: of bf16, four
// pairs of 8 bytes and five CTAs an SM (the same tokens 235 us; eight pairs of 16 bytes 299, two pairs 277, six
// CTAs 313, which spills). Threads that few heads leave over take other tokens: 2 x 30000 tokens, 4 heads of 80 in
// halves 238 us without that, 49; 57835 tokens of 4 heads of 128 90 us and 41.
#include "common.cuh"
#include "serve.h"
#include "sm100.cuh"

namespace s2 {

constexpr int kRopeThreads = 256;

// A CTA takes `tokens` consecutive tokens. Threads x: the units of a head row; threads y: `rows` heads of
// one token or, when that is not all of them, of several.
// A unit is V channels (interleaved), V pairs (half), or V channels beyond `rot`; V = 16 bytes
// (8 for bf16 halves) where strides and widths allow it, else one pair. kVector: every unit starts on a
// multiple of its own 8 or 16 bytes; else its elements are taken one by one.
template <typename T, int V, bool kVector>
__device__ __forceinline__ void load_v(const T* p, float (&x)[V]) {
  if constexpr (kVector && V * sizeof(T) == 16) {
    const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(p));
    const T* y = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = to_f32<T>(y[i]);
  } else if constexpr (kVector && V * sizeof(T) == 8) {
    const uint2 raw = __ldcs(reinterpret_cast<const uint2*>(p));
    const T* y = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = to_f32<T>(y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = to_f32<T>(p[i]);
  }
}
template <typename T, int V, bool kVector>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
  if constexpr (kVector && V * sizeof(T) == 16) {
    uint4 raw;
    T* y = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; i++) y[i] = from_f32<T>(x[i]);
    __stcs(reinterpret_cast<uint4*>(p), raw);
  } else if constexpr (kVector && V * sizeof(T) == 8) {
    uint2 raw;
    T* y = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; i++) y[i] = from_f32<T>(x[i]);
    __stcs(reinterpret_cast<uint2*>(p), raw);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) p[i] = from_f32<T>(x[i]);
  }
}

// One of q and k: the heads of a token that this thread takes, with its (cos, sin) in registers.
template <typename T, int V, bool kHalf, bool kVector, int kPairs>
__device__ __forceinline__ void rotate_heads(const T* src, T* dst, long long is, long long os, int heads, int first,
                                             int step, int pairs, int at, bool rotated, const float2 (&cs)[kPairs]) {
  using namespace sm100;
  constexpr int X = kHalf ? 2 : 1;  // runs of V channels of a unit: one of each half, or one
  src += at;
  dst += at;
  for (int h = first; h < heads; h += step) {
    float x[X][V];
    load_v<T, V, kVector>(src + h * is, x[0]);
    if (kHalf && rotated) load_v<T, V, kVector>(src + h * is + pairs, x[X - 1]);
    if (rotated) {
#pragma unroll
      for (int e = 0; e < kPairs; e++) {
        float& a = kHalf ? x[0][e % V] : x[0][(2 * e) % V];
        float& b = kHalf ? x[X - 1][e % V] : x[0][(2 * e + 1) % V];
        const uint64_t y = ffma2(f2pack(a, b), f2pack(cs[e].x, cs[e].x), fmul2(f2pack(b, a), f2pack(-cs[e].y, cs[e].y)));
        f2unpack(y, a, b);
      }
    }
    store_v<T, V, kVector>(dst + h * os, x[0]);
    if (kHalf && rotated) store_v<T, V, kVector>(dst + h * os + pairs, x[X - 1]);
  }
}

template <typename T, int V, bool kHalf, bool kVector>
__global__ void __launch_bounds__(kRopeThreads, !kHalf ? 8 : V == 4 && sizeof(T) == 2 ? 5 : 6)
    rope_kernel(const __grid_constant__ RopeArgs a, int tokens, int rows) {
  extern __shared__ float2 cs[];  // [tokens][rot / 2]
  constexpr int kPairs = kHalf ? V : V / 2;
  const int pairs = a.rot / 2;
  const long long T0 = (long long)blockIdx.x * tokens;
  const int nt = (int)min((long long)tokens, (long long)a.B * a.N - T0);
  const int b0 = (int)(T0 / a.N), n0 = (int)(T0 - (long long)b0 * a.N);
  for (int e = threadIdx.y * blockDim.x + threadIdx.x; e < nt * pairs; e += blockDim.x * blockDim.y) {
    const int t = e / pairs, i = e - t * pairs;
    int b = b0, n = n0 + t;
    while (n >= a.N) {
      n -= a.N;
      b++;
    }
    const long long at = b * a.ps[0] + n * a.ps[1];
    const double m = a.pos64 ? (double)static_cast<const long long*>(a.pos)[at]
                             : (double)static_cast<const int*>(a.pos)[at];
    const double turn = m * a.turns[i];
    float sn, c;
    sincospif(2.f * (float)(turn - rint(turn)), &sn, &c);
    cs[e] = make_float2(a.mscale * c, a.inverse ? -a.mscale * sn : a.mscale * sn);
  }
  __syncthreads();

  // units of a head row: the rotated ones first, then those that pass through
  const int rot_units = pairs / kPairs, units = rot_units + (a.d - a.rot) / V;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    const bool rotated = u < rot_units;
    const int at = rotated ? u * (kHalf ? kPairs : V) : a.rot + (u - rot_units) * V;
    const int first = threadIdx.y % rows, apart = blockDim.y / rows;  // the thread's first head; its tokens' distance
    for (int t = threadIdx.y / rows; t < nt; t += apart) {
      int b = b0, n = n0 + t;
      while (n >= a.N) {
        n -= a.N;
        b++;
      }
      float2 mine[kPairs];
#pragma unroll
      for (int e = 0; e < kPairs; e++) mine[e] = rotated ? cs[t * pairs + u * kPairs + e] : make_float2(1.f, 0.f);
      rotate_heads<T, V, kHalf, kVector, kPairs>(static_cast<const T*>(a.q) + b * a.qs[0] + n * a.qs[1],
                                               static_cast<T*>(a.qo) + b * a.qos[0] + n * a.qos[1], a.qs[2], a.qos[2],
                                               a.Hq, first, rows, pairs, at, rotated, mine);
      if (a.k)
        rotate_heads<T, V, kHalf, kVector, kPairs>(static_cast<const T*>(a.k) + b * a.ks[0] + n * a.ks[1],
                                                 static_cast<T*>(a.ko) + b * a.kos[0] + n * a.kos[1], a.ks[2], a.kos[2],
                                                 a.Hkv, first, rows, pairs, at, rotated, mine);
    }
  }
}

template <typename T, int V, bool kHalf, bool kVector>
static cudaError_t go(const RopeArgs& a, cudaStream_t st) {
  const long long tokens = (long long)a.B * a.N;
  const int units = (kHalf ? a.rot / 2 / V : a.rot / V) + (a.d - a.rot) / V;
  const int wide = units < 32 ? units : 32, most = kRopeThreads / wide;
  const int heads = a.k && a.Hkv > a.Hq ? a.Hkv : a.Hq, rows = heads < most ? heads : most, apart = most / rows;
  // few heads: the threads that are left take other tokens
  long long tile = tokens < 4 * 592 ? 1 : apart < 4 ? 4 : apart < tokens / 592 ? apart : tokens / 592;
  while (tile > 4 && tile * a.rot / 2 * sizeof(float2) > 16384) tile /= 2;
  const dim3 block(wide, rows * apart);
  rope_kernel<T, V, kHalf, kVector><<<dim3((unsigned)((tokens + tile - 1) / tile)), block, tile * a.rot / 2 * sizeof(float2), st>>>(
      a, (int)tile, rows);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t go_type(const RopeArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T), H = V < 4 ? V : 4;
  // wide units need every row and every run of channels to start and end on one
  // (the pointers do); a unit of the half layout is V pairs, so its halves must too
  const auto multiples = [&a](int unit) {
    bool all = a.d % unit == 0;
    for (int i = 0; i < 3; i++) all = all && a.qs[i] % unit == 0 && (!a.k || a.ks[i] % unit == 0);
    return all;
  };
  const bool wide = multiples(a.half ? H : V) && a.rot % (a.half ? 2 * H : V) == 0;
  if (a.half) return wide ? go<T, H, true, true>(a, st) : go<T, 1, true, false>(a, st);
  if (wide) return go<T, V, false, true>(a, st);
  // One pair a unit: of fp32 that is 8 bytes, one access if all rows start on 8 bytes (those of dense tensors
  // do, as d is even); strides may be odd.
  if constexpr (sizeof(T) == 4)
    if (multiples(2)) return go<T, 2, false, true>(a, st);
  return go<T, 2, false, false>(a, st);
}

cudaError_t launch_rope(const RopeArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? go_type<__nv_bfloat16>(a, st) : go_type<float>(a, st);
}

}  // namespace s2
