// Rows of the 4-bit cache: append (quantise k, v into their slots) and read (the values that
// slots hold).
//
// A group of 32 channels of a token's head is held as fp16 scale = (max - min) / 15 and fp16
// minimum, and codes rint((x - min) / scale) within 0..15, all in IEEE fp32 with the two
// parameters as rounded, so that their rounding costs range at the ends and no bias. Inputs
// are first limited to fp16's range. A NaN or infinity in the k or v of a token's head
// poisons that (token, head): its k scales are NaN, so that every query that attends to it
// gets NaN, and its v is held as zeros, so that queries that do not are left alone.
//
// Bound by HBM: 2 (or 4) bytes a value in, 5/8 byte out. A team of 8..32 lanes takes a token's
// head, k and v at once, eight channels a lane (a 16-byte load of bf16); a group is four
// lanes, its extremes two shuffles away.
#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"

namespace s2 {

constexpr int kRowThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Lanes of a team, and chunks of eight channels (k's, then v's) of each lane.
constexpr int team_lanes(int d) { return d <= 32 ? 8 : d <= 64 ? 16 : 32; }

template <typename T, int TEAM, int CH>
__global__ void __launch_bounds__(kRowThreads) cache4_append_kernel(const __grid_constant__ RowsArgs a) {
  const int lane = threadIdx.x % TEAM;
  const long long rows = (long long)a.T * a.Hkv;
  const long long stride = (long long)gridDim.x * (kRowThreads / TEAM);
  const unsigned mask = TEAM == 32 ? 0xffffffffu
                                   : ((1u << (TEAM & 31)) - 1) << (threadIdx.x % 32 / TEAM * TEAM);
  const int d = a.d, n = d / 32, per = d / 8;  // chunks of k, and of v
  for (long long r = (long long)blockIdx.x * (kRowThreads / TEAM) + threadIdx.x / TEAM; r < rows;
       r += stride) {
    const int t = (int)(r / a.Hkv), h = (int)(r - (long long)t * a.Hkv);
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) continue;  // the team's lanes agree
    float x[CH][8];
    bool bad = false;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      const int ch = lane + c * TEAM;
      if (ch < 2 * per) {
        const bool is_k = ch < per;
        load8<T>(static_cast<const T*>(is_k ? a.k : a.v) + t * (is_k ? a.ks[0] : a.vs[0]) +
                     h * (is_k ? a.ks[1] : a.vs[1]) + (is_k ? ch : ch - per) * 8,
                 x[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) x[c][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; i++) bad |= !(fabsf(x[c][i]) <= 3.402823466e38f);
    }
    bad = __any_sync(mask, bad);
    uint8_t* sub = a.cache + c4::sub_of_slot(slot, h, a.Hkv, a.page_shift, d);
    const int u = slot & 15, row = c4::v_row(u);
#pragma unroll
    for (int c = 0; c < CH; c++) {
      const int ch = lane + c * TEAM;
      const bool is_k = ch < per;
      const int cc = is_k ? ch : ch - per, j = cc >> 2;
      float lo = 65504.f, hi = -65504.f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        // a NaN becomes a limit here; the scale below marks it
        x[c][i] = fminf(fmaxf(x[c][i], -65504.f), 65504.f);
        lo = fminf(lo, x[c][i]);
        hi = fmaxf(hi, x[c][i]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
      }
      __half scale = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
      __half low = __float2half_rn(lo);
      const float s = __half2float(scale), m = __half2float(low);
      uint32_t word = 0;
      if (s > 0.f && !bad) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float q = rintf(__fdiv_rn(__fsub_rn(x[c][i], m), s));
          word |= (uint32_t)fminf(fmaxf(q, 0.f), 15.f) << (4 * i);
        }
      }
      if (bad) {
        scale = is_k ? __ushort_as_half(0x7e00) : __ushort_as_half(0);
        low = __ushort_as_half(0);
      }
      if (ch >= 2 * per) continue;
      if (is_k) {
        *reinterpret_cast<uint32_t*>(sub + c4::k_word(u, j, cc & 3, n)) = word;
        if ((cc & 3) == 0) {
          *reinterpret_cast<__half*>(sub + c4::ks_at(d) + (u * n + j) * 2) = scale;
          *reinterpret_cast<__half*>(sub + c4::km_at(d) + (u * n + j) * 2) = low;
        }
      } else {
        uint8_t* vc = sub + c4::vc_at(d);
        const int g = 2 * (cc & 3);
        *reinterpret_cast<uint16_t*>(vc + c4::v_piece(row, j, g, n)) = (uint16_t)word;
        *reinterpret_cast<uint16_t*>(vc + c4::v_piece(row, j, g + 1, n)) = (uint16_t)(word >> 16);
        if ((cc & 3) == 0)
          *reinterpret_cast<__half2*>(sub + c4::vp_at(d) + (row * n + j) * 4) =
              __halves2half2(scale, low);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
  uint4 raw;
  __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(&raw);
#pragma unroll
  for (int i = 0; i < 8; i++) y[i] = __float2bfloat16_rn(x[i]);
  *reinterpret_cast<uint4*>(p) = raw;
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Values that slots hold; rows of slots outside the cache are zeros, poisoned ones NaN.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) cache4_read_kernel(const __grid_constant__ RowsArgs a) {
  const int d = a.d, n = d / 32, per = d / 8;
  const long long items = (long long)a.T * a.Hkv * 2 * per;
  const long long stride = (long long)gridDim.x * kRowThreads;
  for (long long e = (long long)blockIdx.x * kRowThreads + threadIdx.x; e < items; e += stride) {
    const int ch = (int)(e % (2 * per));
    const long long r = e / (2 * per);
    const int t = (int)(r / a.Hkv), h = (int)(r - (long long)t * a.Hkv);
    const bool is_k = ch < per;
    const int cc = is_k ? ch : ch - per, j = cc >> 2;
    const int slot = a.slots[t];
    float y[8];
    if (slot < 0 || slot >= a.n_slots) {
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = 0.f;
    } else {
      const uint8_t* sub = a.cache + c4::sub_of_slot(slot, h, a.Hkv, a.page_shift, d);
      const int u = slot & 15, row = c4::v_row(u);
      float s = __half2float(
          *reinterpret_cast<const __half*>(sub + c4::ks_at(d) + (u * n + j) * 2));
      float m;
      uint32_t word;
      if (is_k) {
        m = __half2float(*reinterpret_cast<const __half*>(sub + c4::km_at(d) + (u * n + j) * 2));
        word = *reinterpret_cast<const uint32_t*>(sub + c4::k_word(u, j, cc & 3, n));
      } else {
        const __half2 p = *reinterpret_cast<const __half2*>(sub + c4::vp_at(d) + (row * n + j) * 4);
        const bool bad = s != s;
        s = bad ? s : __low2float(p);
        m = __high2float(p);
        const uint8_t* vc = sub + c4::vc_at(d);
        const int g = 2 * (cc & 3);
        word = *reinterpret_cast<const uint16_t*>(vc + c4::v_piece(row, j, g, n)) |
               (uint32_t) * reinterpret_cast<const uint16_t*>(vc + c4::v_piece(row, j, g + 1, n)) << 16;
      }
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = fmaf((float)((word >> (4 * i)) & 15u), s, m);
    }
    store8<T>(static_cast<T*>(is_k ? a.ko : a.vo) + ((size_t)t * a.Hkv + h) * d + cc * 8, y);
  }
}

static unsigned row_blocks(long long threads) {
  const long long blocks = (threads + kRowThreads - 1) / kRowThreads;
  return (unsigned)(blocks > 148 * 8 ? 148 * 8 : blocks);
}

template <typename T>
static cudaError_t append_type(const RowsArgs& a, cudaStream_t st) {
  const long long rows = (long long)a.T * a.Hkv;
  const unsigned grid = row_blocks(rows * team_lanes(a.d));
  if (a.d <= 32)
    cache4_append_kernel<T, 8, 1><<<grid, kRowThreads, 0, st>>>(a);
  else if (a.d <= 64)
    cache4_append_kernel<T, 16, 1><<<grid, kRowThreads, 0, st>>>(a);
  else if (a.d <= 128)
    cache4_append_kernel<T, 32, 1><<<grid, kRowThreads, 0, st>>>(a);
  else
    cache4_append_kernel<T, 32, 2><<<grid, kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache4_append(const RowsArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? append_type<__nv_bfloat16>(a, st) : append_type<float>(a, st);
}

cudaError_t launch_cache4_read(const RowsArgs& a, bool bf16, cudaStream_t st) {
  const unsigned grid = row_blocks((long long)a.T * a.Hkv * (a.d / 4));
  if (bf16)
    cache4_read_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, st>>>(a);
  else
    cache4_read_kernel<float><<<grid, kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace s2
