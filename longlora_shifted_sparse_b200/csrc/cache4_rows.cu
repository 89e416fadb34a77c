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
// A scale whose top value would round beyond fp16's range is taken one step smaller, so that
// readers may form values in fp16.
//
// Bound by HBM: 2 (or 4) bytes a value in, 5/8 byte out, and not far from it by instructions,
// about 15 a value. A team of lanes takes a token, k and v at once, eight channels a lane (a
// 16-byte load of bf16) and kHeads heads in flight; a group is four lanes, its extremes two
// shuffles away. A code is found with the scale's reciprocal and a rounding by addition; a
// quotient that comes within 2^-16 of a border is divided exactly instead.
#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"
#include "sm100.cuh"

namespace s2 {

constexpr int kRowThreads = 256, kHeads = 4;

// Teams: 2 NG groups of four lanes, padded to a power of two; with NG > 4 a lane has two chunks.
constexpr int team_lanes(int ng) { return ng <= 1 ? 8 : ng <= 2 ? 16 : 32; }
constexpr int lane_chunks(int ng) { return ng <= 4 ? 1 : 2; }

template <typename T>
struct Chunk;  // eight values as loaded
template <>
struct Chunk<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { raw = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  // Extremes of the group's four lanes; a NaN comes through.
  __device__ __forceinline__ float2 extremes(unsigned mask) const {
    auto b = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(b(raw.x), b(raw.y)), __hmin2_nan(b(raw.z), b(raw.w)));
    const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(b(raw.x), b(raw.y)), __hmax2_nan(b(raw.z), b(raw.w)));
    const uint32_t l = *reinterpret_cast<const uint32_t*>(&lo), h = *reinterpret_cast<const uint32_t*>(&hi) ^ 0x80008000u;
    const uint32_t p0 = __byte_perm(l, h, 0x5410u), p1 = __byte_perm(l, h, 0x7632u);  // (min, -max) twice
    __nv_bfloat162 e = __hmin2_nan(b(p0), b(p1));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const uint32_t other = __shfl_xor_sync(mask, *reinterpret_cast<const uint32_t*>(&e), o);
      e = __hmin2_nan(e, b(other));
    }
    return make_float2(__low2float(e), -__high2float(e));
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w) : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
  static __device__ __forceinline__ float fmin_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
  }
  static __device__ __forceinline__ float fmax_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
  }
  __device__ __forceinline__ float2 extremes(unsigned mask) const {
    float lo = a.x, hi = a.x;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 y = pair(i);
      lo = fmin_nan(fmin_nan(lo, y.x), y.y);
      hi = fmax_nan(fmax_nan(hi, y.x), y.y);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = fmin_nan(lo, __shfl_xor_sync(mask, lo, o));
      hi = fmax_nan(hi, __shfl_xor_sync(mask, hi, o));
    }
    return make_float2(lo, hi);
  }
};

// Codes of eight values, channel i in bits 4 i. `wide`: some lie beyond fp16.
template <typename T>
__device__ __forceinline__ uint32_t codes8(const Chunk<T>& x, float s, float m, bool wide) {
  using namespace sm100;
  const float inv = __frcp_rn(s);
  const uint64_t m2 = f2pack(-m, -m), inv2 = f2pack(inv, inv), big = f2pack(12582912.f, 12582912.f);  // 1.5 * 2^23
  uint32_t t[8];
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    float2 y = x.pair(i);
    if (wide) {
      y.x = fminf(fmaxf(y.x, -65504.f), 65504.f);
      y.y = fminf(fmaxf(y.y, -65504.f), 65504.f);
    }
    float q0, q1, d0, d1, t0, t1;
    f2unpack(fmul2(fadd2(f2pack(y.x, y.y), m2), inv2), q0, q1);
    q0 = fminf(fmaxf(q0, 0.f), 15.f);
    q1 = fminf(fmaxf(q1, 0.f), 15.f);
    const uint64_t q = f2pack(q0, q1), r = fadd2(q, big);
    f2unpack(fsub2(q, fsub2(r, big)), d0, d1);
    f2unpack(r, t0, t1);
    off = fmax3(off, fabsf(d0), fabsf(d1));
    t[2 * i] = __float_as_uint(t0);
    t[2 * i + 1] = __float_as_uint(t1);
  }
  if (off > 0.5f - 0x1p-16f) {
    // q is within 2^-18 of the rounded quotient (three roundings of a value below 16)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float2 y = x.pair(i);
      y.x = fminf(fmaxf(y.x, -65504.f), 65504.f);
      y.y = fminf(fmaxf(y.y, -65504.f), 65504.f);
      t[2 * i] = 0x4b400000u + (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(y.x, m), s)), 0.f), 15.f);
      t[2 * i + 1] = 0x4b400000u + (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(y.y, m), s)), 0.f), 15.f);
    }
  }
  // the addend's own bits leave the word with the constant, or at its top
  uint32_t word = 0u - (0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8));
#pragma unroll
  for (int i = 0; i < 8; i++) word += t[i] << (4 * i);
  return word;
}

template <typename T, int NG>
__global__ void __launch_bounds__(kRowThreads) cache4_append_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int TEAM = team_lanes(NG), CH = lane_chunks(NG), D = 32 * NG, PER = D / 8;  // chunks of k, and of v
  const int lane = threadIdx.x % TEAM;
  const unsigned mask = TEAM == 32 ? 0xffffffffu : ((1u << (TEAM & 31)) - 1) << (threadIdx.x % 32 / TEAM * TEAM);
  const int t = blockIdx.x * (kRowThreads / TEAM) + threadIdx.x / TEAM, h0 = blockIdx.y * kHeads;
  if (t >= a.T) return;  // whole teams
  const int slot = a.slots[t];
  if (slot < 0 || slot >= a.n_slots) return;
  const int nh = min(kHeads, a.Hkv - h0);
  Chunk<T> x[kHeads][CH];
#pragma unroll
  for (int e = 0; e < kHeads; e++)
#pragma unroll
    for (int c = 0; c < CH; c++) {
      const int ch = lane + c * TEAM;
      const bool is_k = ch < PER;
      if (e < nh && ch < 2 * PER)
        x[e][c].load(static_cast<const T*>(is_k ? a.k : a.v) + t * (is_k ? a.ks[0] : a.vs[0]) +
                     (h0 + e) * (is_k ? a.ks[1] : a.vs[1]) + (is_k ? ch : ch - PER) * 8);
      else
        x[e][c].clear();
    }
  const int u = slot & 15, row = c4::v_row(u);
  uint8_t* sub = a.cache + c4::sub_of_slot(slot, h0, a.Hkv, a.page_shift, D);
  const size_t head_bytes = (size_t)c4::sub_bytes(D) << (a.page_shift - 4);
#pragma unroll
  for (int e = 0; e < kHeads; e++) {
    if (e >= nh) break;
    float2 ex[CH];
    bool bad = false;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      ex[c] = x[e][c].extremes(mask);
      bad |= !(fabsf(ex[c].x) <= 3.402823466e38f && fabsf(ex[c].y) <= 3.402823466e38f);
    }
    bad = __any_sync(mask, bad);
#pragma unroll
    for (int c = 0; c < CH; c++) {
      const int ch = lane + c * TEAM;
      const bool is_k = ch < PER;
      const int cc = is_k ? ch : ch - PER, j = cc >> 2;
      const float lo = fminf(fmaxf(ex[c].x, -65504.f), 65504.f), hi = fminf(fmaxf(ex[c].y, -65504.f), 65504.f);
      __half scale = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
      __half low = __float2half_rn(lo);
      float s = __half2float(scale);
      const float m = __half2float(low);
      if (fmaf(15.f, s, m) >= 65520.f) {  // would round to infinity in fp16
        scale = __ushort_as_half(__half_as_ushort(scale) - 1);
        s = __half2float(scale);
      }
      uint32_t word = 0;
      if (s > 0.f && !bad) word = codes8<T>(x[e][c], s, m, ex[c].x < -65504.f || ex[c].y > 65504.f);
      if (bad) {
        scale = is_k ? __ushort_as_half(0x7e00) : __ushort_as_half(0);
        low = __ushort_as_half(0);
      }
      uint32_t other = 0;
      if (NG % 2 == 0) {  // v: the half-words of two groups lie together; lanes 4 apart swap
        const bool up = j & 1;
        other = __shfl_xor_sync(mask, up ? word & 0xffffu : word >> 16, 4);
      }
      if (ch >= 2 * PER) continue;
      if (is_k) {
        *reinterpret_cast<uint32_t*>(sub + c4::k_word(u, j, cc & 3, NG)) = word;
        if ((cc & 3) == 0) {
          *reinterpret_cast<__half*>(sub + c4::ks_at(D) + (u * NG + j) * 2) = scale;
          *reinterpret_cast<__half*>(sub + c4::km_at(D) + (u * NG + j) * 2) = low;
        }
      } else {
        uint8_t* vc = sub + c4::vc_at(D);
        const int g = 2 * (cc & 3);
        if (NG % 2 == 0) {
          const bool up = j & 1;
          *reinterpret_cast<uint32_t*>(vc + c4::v_piece(row, j & ~1, g + up, NG)) =
              up ? other | (word & 0xffff0000u) : (word & 0xffffu) | other << 16;
        } else {
          *reinterpret_cast<uint16_t*>(vc + c4::v_piece(row, j, g, NG)) = (uint16_t)word;
          *reinterpret_cast<uint16_t*>(vc + c4::v_piece(row, j, g + 1, NG)) = (uint16_t)(word >> 16);
        }
        if ((cc & 3) == 0)
          *reinterpret_cast<__half2*>(sub + c4::vp_at(D) + (row * NG + j) * 4) = __halves2half2(scale, low);
      }
    }
    sub += head_bytes;
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
  __stcs(reinterpret_cast<uint4*>(p), raw);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

// Values that slots hold; rows of slots outside the cache are zeros, poisoned ones NaN. The same
// teams, a chunk of eight values a lane.
template <typename T, int NG>
__global__ void __launch_bounds__(kRowThreads) cache4_read_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int TEAM = team_lanes(NG), CH = lane_chunks(NG), D = 32 * NG, PER = D / 8;
  const int lane = threadIdx.x % TEAM;
  const int t = blockIdx.x * (kRowThreads / TEAM) + threadIdx.x / TEAM, h0 = blockIdx.y * kHeads;
  if (t >= a.T) return;
  const int slot = a.slots[t];
  const bool there = slot >= 0 && slot < a.n_slots;
  const int nh = min(kHeads, a.Hkv - h0), u = slot & 15, row = c4::v_row(u);
  const uint8_t* sub = there ? a.cache + c4::sub_of_slot(slot, h0, a.Hkv, a.page_shift, D) : nullptr;
  const size_t head_bytes = (size_t)c4::sub_bytes(D) << (a.page_shift - 4);
#pragma unroll
  for (int c = 0; c < CH; c++) {
    const int ch = lane + c * TEAM;
    if (ch >= 2 * PER) continue;
    const bool is_k = ch < PER;
    const int cc = is_k ? ch : ch - PER, j = cc >> 2, g = 2 * (cc & 3);
    uint32_t word[kHeads], scale[kHeads], pair[kHeads];
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      word[e] = scale[e] = pair[e] = 0u;
      if (!there || e >= nh) continue;
      const uint8_t* p = sub + e * head_bytes;
      scale[e] = *reinterpret_cast<const uint16_t*>(p + c4::ks_at(D) + (u * NG + j) * 2);
      if (is_k) {
        pair[e] = *reinterpret_cast<const uint16_t*>(p + c4::km_at(D) + (u * NG + j) * 2);
        word[e] = *reinterpret_cast<const uint32_t*>(p + c4::k_word(u, j, cc & 3, NG));
      } else {
        pair[e] = *reinterpret_cast<const uint32_t*>(p + c4::vp_at(D) + (row * NG + j) * 4);
        word[e] = *reinterpret_cast<const uint16_t*>(p + c4::vc_at(D) + c4::v_piece(row, j, g, NG)) |
                  (uint32_t) * reinterpret_cast<const uint16_t*>(p + c4::vc_at(D) + c4::v_piece(row, j, g + 1, NG)) << 16;
      }
    }
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      if (e >= nh) continue;
      float s = __half2float(__ushort_as_half((unsigned short)scale[e]));
      float m = __half2float(__ushort_as_half((unsigned short)pair[e]));
      if (!is_k) {
        s = s != s ? s : m;  // the k scales carry the poison
        m = __half2float(__ushort_as_half((unsigned short)(pair[e] >> 16)));
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = fmaf((float)((word[e] >> (4 * i)) & 15u), s, m);
      store8<T>(static_cast<T*>(is_k ? a.ko : a.vo) + ((size_t)t * a.Hkv + h0 + e) * D + cc * 8, y);
    }
  }
}

template <typename T, int NG>
static void go(const RowsArgs& a, bool append, cudaStream_t st) {
  const int teams = kRowThreads / team_lanes(NG);
  const dim3 grid((unsigned)(((long long)a.T + teams - 1) / teams), (unsigned)((a.Hkv + kHeads - 1) / kHeads));
  if (append)
    cache4_append_kernel<T, NG><<<grid, kRowThreads, 0, st>>>(a);
  else
    cache4_read_kernel<T, NG><<<grid, kRowThreads, 0, st>>>(a);
}

template <typename T>
static cudaError_t go_type(const RowsArgs& a, bool append, cudaStream_t st) {
  switch (a.d / 32) {
    case 1: go<T, 1>(a, append, st); break;
    case 2: go<T, 2>(a, append, st); break;
    case 3: go<T, 3>(a, append, st); break;
    case 4: go<T, 4>(a, append, st); break;
    case 5: go<T, 5>(a, append, st); break;
    case 6: go<T, 6>(a, append, st); break;
    case 7: go<T, 7>(a, append, st); break;
    default: go<T, 8>(a, append, st);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache4_append(const RowsArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? go_type<__nv_bfloat16>(a, true, st) : go_type<float>(a, true, st);
}

cudaError_t launch_cache4_read(const RowsArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? go_type<__nv_bfloat16>(a, false, st) : go_type<float>(a, false, st);
}

}  // namespace s2
