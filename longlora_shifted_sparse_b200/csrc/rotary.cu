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
// are then fp32. They are formed once per (token, pair) of a CTA's tile, in shared memory,
// and shared by all heads: fp64 work per token is rot/2 products.
#include "common.cuh"
#include "serve.h"

namespace s2 {

constexpr int kRopeThreads = 256;

// A CTA takes `tokens` consecutive tokens and one slice of the heads (q's, then k's).
// Threads x: the units of a head row; threads y: rows (token, head), kRows of them in flight.
// A unit is V channels (interleaved), V pairs (half), or V channels beyond `rot`; V = 16 bytes
// where strides and widths allow it, else one pair.
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&x)[V]) {
  if constexpr (V * sizeof(T) == 16) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const T* y = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = to_f32<T>(y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = to_f32<T>(p[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
  if constexpr (V * sizeof(T) == 16) {
    uint4 raw;
    T* y = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; i++) y[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(p) = raw;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) p[i] = from_f32<T>(x[i]);
  }
}

template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                            int tokens, int head_slice) {
  extern __shared__ float2 cs[];  // [tokens][rot / 2]
  const int pairs = a.rot / 2;
  const long long T0 = (long long)blockIdx.x * tokens;
  const int nt = (int)min((long long)tokens, (long long)a.B * a.N - T0);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int e = tid; e < nt * pairs; e += blockDim.x * blockDim.y) {
    const int t = e / pairs, i = e - t * pairs;
    const int b = (int)((T0 + t) / a.N), n = (int)((T0 + t) - (long long)b * a.N);
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
  const int rot_units = kHalf ? pairs / V : a.rot / V;
  const int pass_units = (a.d - a.rot) / V;
  const int heads = a.Hq + (a.k ? a.Hkv : 0);
  const int h_begin = blockIdx.y * head_slice, nh = min(head_slice, heads - h_begin);
  const int rows = nt * nh;
  for (int u = threadIdx.x; u < rot_units + pass_units; u += blockDim.x) {
    for (int r = threadIdx.y; r < rows; r += blockDim.y) {
      const int t = r / nh, hh = h_begin + (r - t * nh);
      const int b = (int)((T0 + t) / a.N), n = (int)((T0 + t) - (long long)b * a.N);
      const bool is_q = hh < a.Hq;
      const int h = is_q ? hh : hh - a.Hq;
      const long long* is = is_q ? a.qs : a.ks;
      const long long* os = is_q ? a.qos : a.kos;
      const T* src = static_cast<const T*>(is_q ? a.q : a.k) + b * is[0] + n * is[1] + h * is[2];
      T* dst = static_cast<T*>(is_q ? a.qo : a.ko) + b * os[0] + n * os[1] + h * os[2];
      if (u >= rot_units) {
        const int x = a.rot + (u - rot_units) * V;
        float y[V];
        load_v<T, V>(src + x, y);
        store_v<T, V>(dst + x, y);
      } else if (kHalf) {
        const int i = u * V;
        float x0[V], x1[V], y0[V], y1[V];
        load_v<T, V>(src + i, x0);
        load_v<T, V>(src + pairs + i, x1);
#pragma unroll
        for (int e = 0; e < V; e++) {
          const float2 c = cs[t * pairs + i + e];
          y0[e] = fmaf(x0[e], c.x, -x1[e] * c.y);
          y1[e] = fmaf(x0[e], c.y, x1[e] * c.x);
        }
        store_v<T, V>(dst + i, y0);
        store_v<T, V>(dst + pairs + i, y1);
      } else {
        float x[V], y[V];
        load_v<T, V>(src + u * V, x);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 c = cs[t * pairs + (u * V + e) / 2];
          y[e] = fmaf(x[e], c.x, -x[e + 1] * c.y);
          y[e + 1] = fmaf(x[e], c.y, x[e + 1] * c.x);
        }
        store_v<T, V>(dst + u * V, y);
      }
    }
  }
}

template <typename T, int V, bool kHalf>
static cudaError_t go(const RopeArgs& a, cudaStream_t st) {
  const long long tokens = (long long)a.B * a.N;
  const int heads = a.Hq + (a.k ? a.Hkv : 0);
  const int units = (kHalf ? a.rot / 2 / V : a.rot / V) + (a.d - a.rot) / V;
  const int tile = tokens >= 4 * 592 ? 4 : 1;
  const dim3 block(units < 32 ? units : 32, kRopeThreads / (units < 32 ? units : 32));
  rope_kernel<T, V, kHalf><<<dim3((unsigned)((tokens + tile - 1) / tile)), block,
                             tile * a.rot / 2 * sizeof(float2), st>>>(a, tile, heads);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t go_type(const RopeArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte units need every row and every run of channels to start and end on 16 bytes
  // (the pointers do); a unit of the half layout is V pairs, so its halves must too
  bool wide = a.d % V == 0 && a.rot % (a.half ? 2 * V : V) == 0;
  for (int i = 0; i < 3; i++) wide = wide && a.qs[i] % V == 0 && (!a.k || a.ks[i] % V == 0);
  if (a.half)
    return wide ? go<T, V, true>(a, st) : go<T, 1, true>(a, st);
  return wide ? go<T, V, false>(a, st) : go<T, 2, false>(a, st);
}

cudaError_t launch_rope(const RopeArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? go_type<__nv_bfloat16>(a, st) : go_type<float>(a, st);
}

}  // namespace s2
