// Rows of the 4-bit cache: append (quantise k, v into their slots) and read (the values that
// slots hold).
//
// A group of 32 channels of a token's head is held as fp16 scale = (max - min) * (1 / 15) and fp16
// minimum, and codes rint((x - min) / scale) within 0..15, all in IEEE fp32 with the two
// parameters as rounded, so that their rounding costs range at the ends and no bias. Inputs
// are first limited to fp16's range. A NaN or infinity in the k or v of a token's head
// poisons that (token, head): its k scales are NaN, so that every query that attends to it
// gets NaN, and its v is held as zeros, so that queries that do not are left alone.
//
// A scale whose top value would round beyond fp16's range is taken one step smaller, so that
// readers may form values in fp16.
//
// Bound by HBM: 2 (or 4) bytes a value in, 5/8 byte out, with instructions not far behind. To
// append, a lane takes a whole group, so that its extremes, scale and reciprocal are found once and
// without shuffles (a lane for eight channels, four to a group, took three times the
// instructions and 258 us for 32768 tokens of 32 heads of 128). A code is found with the scale's
// reciprocal, a step with the residual that makes the quotient the rounded one, and a rounding by
// addition. To read, a lane takes eight channels, so that stores are whole lines. 32768 tokens, 32 heads of 128,
// bf16: append 168 us (705 MB, 4.2 TB/s), read 150 us (4.7 TB/s).
#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"
#include "sm100.cuh"

namespace s2 {

constexpr int kRowThreads = 256;

template <typename T>
struct Chunk;  // eight values as loaded
template <>
struct Chunk<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float value(int i) const {  // i known at compile time
    const uint32_t w = i < 2 ? raw.x : i < 4 ? raw.y : i < 6 ? raw.z : raw.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  // Extremes of four chunks; a NaN comes through.
  static __device__ __forceinline__ float2 extremes(const Chunk (&x)[4]) {
    auto b = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 lo = b(x[0].raw.x), hi = lo;
#pragma unroll
    for (int c = 0; c < 4; c++) {
      lo = __hmin2_nan(__hmin2_nan(lo, b(x[c].raw.x)), __hmin2_nan(__hmin2_nan(b(x[c].raw.y), b(x[c].raw.z)), b(x[c].raw.w)));
      hi = __hmax2_nan(__hmax2_nan(hi, b(x[c].raw.x)), __hmax2_nan(__hmax2_nan(b(x[c].raw.y), b(x[c].raw.z)), b(x[c].raw.w)));
    }
    return make_float2(__bfloat162float(__hmin_nan(lo.x, lo.y)), __bfloat162float(__hmax_nan(hi.x, hi.y)));
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ float value(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
  static __device__ __forceinline__ float2 extremes(const Chunk (&x)[4]) {
    float lo = x[0].a.x, hi = lo;
#pragma unroll
    for (int c = 0; c < 4; c++)
#pragma unroll
      for (int i = 0; i < 8; i++) {
        asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(x[c].value(i)));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(x[c].value(i)));
      }
    return make_float2(lo, hi);
  }
};

// Codes of eight values, channel i in bits 4 i, of values whose quotients lie within -0.5 .. 15.5.
// The quotient is (x - m) inv and a step with its residual, which makes it the correctly rounded one, as inv is the correctly
// rounded reciprocal (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
template <typename T>
__device__ __forceinline__ uint32_t codes8(const Chunk<T>& x, uint64_t minus_m, uint64_t minus_s, uint64_t inv) {
  using namespace sm100;
  const uint64_t big = f2pack(12582912.f, 12582912.f), minus_big = f2pack(-12582912.f, -12582912.f);  // 1.5 * 2^23
  // channels i and i + 4 at once; their codes gather in the low 16 bits of two floats, exactly
  uint64_t acc = big;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint64_t y = fadd2(f2pack(x.value(i), x.value(i + 4)), minus_m), q = fmul2(y, inv);
    const uint64_t r = fadd2(fadd2(ffma2(ffma2(q, minus_s, y), inv, q), big), minus_big);
    const float unit = (float)(1 << (4 * i));
    acc = ffma2(r, f2pack(unit, unit), acc);
  }
  float w0, w1;
  f2unpack(acc, w0, w1);
  return __byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x5410u);
}
// The same by the division itself, for inputs anywhere.
template <typename T>
__device__ __noinline__ uint32_t codes8_exact(Chunk<T> x, float m, float s) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float y = fminf(fmaxf(x.value(i), -65504.f), 65504.f);
    word |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(y, m), s)), 0.f), 15.f) << (4 * i);
  }
  return word;
}

// A team of 2 NG lanes takes a token's head: the groups of k, then those of v.
template <typename T, int NG>
__global__ void __launch_bounds__(kRowThreads) cache4_append_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int TEAM = 2 * NG, TEAMS = 32 / TEAM, D = 32 * NG;
  const int lane = threadIdx.x & 31, team = lane / TEAM, in = lane % TEAM;
  const bool is_k = in < NG;
  const int j = is_k ? in : in - NG;
  const long long r = ((long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * TEAMS + team;
  const bool live = team < TEAMS && r < (long long)a.T * a.Hkv;
  const int t = live ? (int)((unsigned)r / (unsigned)a.Hkv) : 0, h = live ? (int)r - t * a.Hkv : 0;
  const int slot = live ? a.slots[t] : -1;
  const bool stored = slot >= 0 && slot < a.n_slots;
  Chunk<T> x[4];
  const T* p = static_cast<const T*>(is_k ? a.k : a.v) + t * (is_k ? a.ks[0] : a.vs[0]) + h * (is_k ? a.ks[1] : a.vs[1]) + 32 * j;
#pragma unroll
  for (int c = 0; c < 4; c++) x[c].load(p + 8 * c);  // (dead lanes: the first row)
  const float2 ex = Chunk<T>::extremes(x);
  const unsigned bads =
      __ballot_sync(0xffffffffu, !(fabsf(ex.x) <= 3.402823466e38f && fabsf(ex.y) <= 3.402823466e38f));
  const bool bad = (bads >> (team * TEAM)) & ((2u << (TEAM - 1)) - 1u);
  const float lo = fminf(fmaxf(ex.x, -65504.f), 65504.f), hi = fminf(fmaxf(ex.y, -65504.f), 65504.f);
  __half low = __float2half_rn(lo);
  __half scale = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 0.0666666701f));  // 1 / 15
  float s = __half2float(scale);
  const float m = __half2float(low);
  if (fmaf(15.f, s, m) >= 65520.f) {  // would round to infinity in fp16
    scale = __ushort_as_half(__half_as_ushort(scale) - 1);
    s = __half2float(scale);
  }
  uint32_t word[4] = {0u, 0u, 0u, 0u};
  if (s > 0.f && !bad) {
    const float inv = __frcp_rn(s);
    // A value may lie outside the codes' range where the group's minimum is far from its fp16
    // neighbour, for the group's width, or where some input is beyond fp16.
    if ((lo - m) * inv < -0.49f || (hi - m) * inv > 15.49f || ex.x != lo || ex.y != hi) {
#pragma unroll
      for (int c = 0; c < 4; c++) word[c] = codes8_exact<T>(x[c], m, s);
    } else {
      const uint64_t minus_m = sm100::f2pack(-m, -m), minus_s = sm100::f2pack(-s, -s), inv2 = sm100::f2pack(inv, inv);
#pragma unroll
      for (int c = 0; c < 4; c++) word[c] = codes8<T>(x[c], minus_m, minus_s, inv2);
    }
  }
  if (bad) {
    scale = is_k ? __ushort_as_half(0x7e00) : __ushort_as_half(0);
    low = __ushort_as_half(0);
  }
  const int u = slot & 15, row = c4::v_row(u);
  uint8_t* sub = a.cache + c4::sub_of_slot(stored ? slot : 0, h, a.Hkv, a.page_shift, D);
  const bool up = j & 1;
#pragma unroll
  for (int c = 0; c < 4; c++) {
    if (NG % 2 == 0) {  // v: the half-words of two groups lie together; their lanes swap
      const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? word[c] & 0xffffu : word[c] >> 16, 1);
      const uint32_t swapped = __byte_perm(word[c], other, up ? 0x3254u : 0x5410u);
      const int at = is_k ? c4::k_word(u, j, c, NG) : c4::vc_at(D) + c4::v_piece(row, j & ~1, 2 * c + up, NG);
      if (stored) *reinterpret_cast<uint32_t*>(sub + at) = is_k ? word[c] : swapped;
    } else if (stored) {
      if (is_k) {
        *reinterpret_cast<uint32_t*>(sub + c4::k_word(u, j, c, NG)) = word[c];
      } else {
        *reinterpret_cast<uint16_t*>(sub + c4::vc_at(D) + c4::v_piece(row, j, 2 * c, NG)) = (uint16_t)word[c];
        *reinterpret_cast<uint16_t*>(sub + c4::vc_at(D) + c4::v_piece(row, j, 2 * c + 1, NG)) = (uint16_t)(word[c] >> 16);
      }
    }
  }
  if (stored) {
    const int at = is_k ? c4::ks_at(D) + (u * NG + j) * 2 : c4::vp_at(D) + (row * NG + j) * 4;
    *reinterpret_cast<__half*>(sub + at) = scale;
    *reinterpret_cast<__half*>(sub + (is_k ? c4::km_at(D) + (u * NG + j) * 2 : at + 2)) = low;
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

// Values that slots hold; rows of slots outside the cache are zeros, poisoned ones NaN. Teams of
// lanes take a token and kHeads heads in flight: the chunks of eight channels of k, then of v, padded
// to a power of two; with NG > 4 a lane has two.
constexpr int kHeads = 4;
constexpr int team_lanes(int ng) { return ng <= 1 ? 8 : ng <= 2 ? 16 : 32; }
constexpr int lane_chunks(int ng) { return ng <= 4 ? 1 : 2; }

template <typename T, int NG>
__global__ void __launch_bounds__(kRowThreads) cache4_read_kernel(const __grid_constant__ RowsArgs a) {
  using namespace sm100;
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
    const uint8_t* at_word = sub + (is_k ? c4::k_word(u, j, cc & 3, NG) : c4::vc_at(D) + c4::v_piece(row, j, g, NG));
    const int next = is_k ? 2 : c4::v_piece(row, j, g + 1, NG) - c4::v_piece(row, j, g, NG);
    const uint8_t* at_scale = sub + c4::ks_at(D) + (u * NG + j) * 2;  // of v too: it carries the poison
    const uint8_t* at_pair = sub + (is_k ? c4::km_at(D) + (u * NG + j) * 2 : c4::vp_at(D) + (row * NG + j) * 4);
    uint32_t word[kHeads], scale[kHeads], pair[kHeads];
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      word[e] = scale[e] = pair[e] = 0u;
      if (!there || e >= nh) continue;
      word[e] = *reinterpret_cast<const uint16_t*>(at_word + e * head_bytes) |
                (uint32_t) * reinterpret_cast<const uint16_t*>(at_word + e * head_bytes + next) << 16;
      scale[e] = *reinterpret_cast<const uint16_t*>(at_scale + e * head_bytes);
      pair[e] = is_k ? *reinterpret_cast<const uint16_t*>(at_pair + e * head_bytes)
                     : *reinterpret_cast<const uint32_t*>(at_pair + e * head_bytes);
    }
    T* out = static_cast<T*>(is_k ? a.ko : a.vo) + ((size_t)t * a.Hkv + h0) * D + cc * 8;
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      if (e >= nh) continue;
      float s = __half2float(__ushort_as_half((unsigned short)scale[e]));
      float m = __half2float(__ushort_as_half((unsigned short)pair[e]));
      if (!is_k) {
        s = s != s ? s : m;
        m = __half2float(__ushort_as_half((unsigned short)(pair[e] >> 16)));
      }
      // A code in bits 4 i of 2^23 is 16^i times itself; the power goes into the scale. Channels i and
      // i + 4 at once, those of the upper half from the word's upper half.
      const uint32_t high = word[e] >> 16;
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t mask = 15u << (4 * i);
        const uint64_t code = fadd2(f2pack(__uint_as_float((word[e] & mask) | 0x4b000000u), __uint_as_float((high & mask) | 0x4b000000u)),
                                    f2pack(-8388608.f, -8388608.f));
        const float unit = s * (1.f / (1 << (4 * i)));
        f2unpack(ffma2(code, f2pack(unit, unit), f2pack(m, m)), y[i], y[i + 4]);
      }
      store8<T>(out + (size_t)e * D, y);
    }
  }
}

template <typename T, int NG>
static void go(const RowsArgs& a, bool append, cudaStream_t st) {
  if (append) {
    constexpr int rows = kRowThreads / 32 * (32 / (2 * NG));
    cache4_append_kernel<T, NG><<<(unsigned)(((long long)a.T * a.Hkv + rows - 1) / rows), kRowThreads, 0, st>>>(a);
  } else {
    constexpr int teams = kRowThreads / team_lanes(NG);
    const dim3 grid((unsigned)(((long long)a.T + teams - 1) / teams), (unsigned)((a.Hkv + kHeads - 1) / kHeads));
    cache4_read_kernel<T, NG><<<grid, kRowThreads, 0, st>>>(a);
  }
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
