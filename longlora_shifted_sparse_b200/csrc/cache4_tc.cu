// Attention over the 4-bit cache for many query rows at once (chunks of prompts), on the
// 5th-generation tensor cores.
//
// O = softmax(Q K^T * scale) V for tiles of 256 query rows of one (request, kv head): the heads
// that share it, times the request's tokens, in two MMA tiles of 128 rows (A, B) that share every
// dequantised key and value. Bound by the tensor cores and, at their speed, by the softmax and
// the dequantisation beside them; the cache's own bytes are read once per 256 rows.
//
// Roles (640 threads):
//   warp 0        MMA issuer and TMEM owner (warps 1..3 complete its warpgroup, whose registers go to
//                 the others). Per tile of 128 keys: PV_A(j-1), QK_A(j), PV_B(j-1), QK_B(j), so that one
//                 tile's softmax runs under the other's MMAs; steps run on across units.
//   warps 4..11   copies and dequantisation, sixteen tokens of every tile each: their k (or v) is one
//                 contiguous piece of 10 d bytes, copied a tile ahead by cp.async; then
//                 minimum + scale * code in fp16 is written as the MMAs' 128-byte-swizzled operands (K
//                 rows of channels; V the same, read by the MMA transposed), K of tile j with V of
//                 tile j - 1. Channels lie in the order 0 4 1 5 2 6 3 7 within each eight, the order in
//                 which two codes come out of a word together: Q, which they bring to fp16 too, is
//                 written in the same order, and O is put right when it is stored.
//   warps 12..19  softmax and O, a thread a row (TMEM lane).
// fp16 holds k and v to half a step 2^-11 of the value (the codes are 4 bits wide) and P to 2^-11
// of itself, below the output's bf16 (2^-8); scores, maxima, sums and O are fp32.
// The running maximum is kept as an integer 8 below the row's first ones (P then uses fp16's range: it is
// dropped below 2^-33 of them) and moves only when a sum of P shows that some P might leave that range, so that the common
// step takes no maximum and O is rescaled, exactly, a few times a row.
//
// Work is steps of 128 keys, laid on one line over (request, kv head, tile) with the steps that the
// tile's last row sees; every CTA takes an equal run of the line. A tile that several CTAs share
// leaves parts (sums and maxima in fp32) that a second launch joins in the order of the runs.
// Every wait is bounded; on expiry the status word is set and the CTA drains.
//
// Measured (B200, 64 heads on 8 of 128, 512 tokens over 32768): 575 us, 950 TFLOP/s; two requests over 16384
// and 8636: 421 to 448 us from one GPU to another, 800 to 850. What was tried: mma.sync in tiles of 32 rows 2015 us; three dequantising
// warps 735, seven 486 (16 softmax warps), a thread a row without the maximum 440; bulk copies
// instead of cp.async 467 (4700 cycles to arrive beside the MMAs' operand reads); 16 softmax warps
// 486; PV in two halves of the keys, the first under the second's softmax, 500. The MMAs of a half step
// take ~1900 cycles of ~2170 (1024 of tensor work).
#include <math.h>

#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"
#include "sm100.cuh"

namespace s2 {
namespace {

using namespace sm100;

constexpr int kRows = 128, kKeys = 128;
// Warps: the issuer and three idle ones, eight that fill, eight of the softmax. Five share one
// scheduler's registers, so a launch hands each thread 96; then they are split (setmaxnreg).
constexpr int kFill0 = 4, kFillWarps = 8, kSoft0 = 12, kThreads = 640;
constexpr int kRegsIssue = 40, kRegsFill = 88, kRegsSoftmax = 128;
static_assert(kRegsIssue + 2 * kRegsFill + 2 * kRegsSoftmax <= 5 * 96, "register split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;
// log2 units. A P of a new maximum is at most 2^kBelow, so that 64 of them stay within kSumLimit, and where their sum
// does not, the largest is above 2^kGrow: the maximum moves.
constexpr float kBelow = 8.f, kGrow = 9.f;
constexpr float kSumLimit = 60000.f;          // no P of such a sum overflows fp16
// A maximum of this size or more is taken as it is, and its row goes the long way: 8 below it is no longer a number of its own, and
// a product that is not rounded before the maximum is taken off would be away from it by more than fp16 spans.
constexpr float kLarge = 0x1p22f;

template <int D>
struct Layout {
  static constexpr uint32_t tile = kKeys * D * 2;       // an operand tile of 128 rows
  static constexpr uint32_t half = kKeys * 128;         // its first 64 channels
  static constexpr uint32_t piece = 10 * D;             // 16 tokens of k, or of v
  static constexpr uint32_t q = 0, k = 2 * tile, v = 4 * tile, ring = 6 * tile;
  static constexpr uint32_t bytes = ring + 2 * kFillWarps * piece + 1024;
};

// The line of work: requests in order; in a request kv heads, then tiles of 256 rows, then steps.
struct Walk {
  int group, r, row0, n, held, tiles, h, t;
  int q, rem;          // ((t + 1) * 256 - 1) divided by group: the tile's last token, unless it is cut

  __device__ __forceinline__ void request(const Cache4AttnArgs& a, int at) {
    r = at;
    const int begin = a.cu[r], end = a.cu[r + 1];
    row0 = begin;
    n = begin >= 0 && end > begin && end <= a.T ? end - begin : 0;
    held = (int)min((long long)max(a.lens[r], 0), (long long)a.max_pages << a.page_shift);
    tiles = (int)(((long long)n * group + 2 * kRows - 1) / (2 * kRows));
    first_tile();
  }
  __device__ __forceinline__ void first_tile() {
    t = 0;
    q = (2 * kRows - 1) / group;
    rem = (2 * kRows - 1) - q * group;
  }
  __device__ __forceinline__ void next_tile() {
    t++;
    q += (2 * kRows) / group;
    rem += (2 * kRows) % group;
    if (rem >= group) {
      rem -= group;
      q++;
    }
  }
  __device__ __forceinline__ int sees() const {  // keys of the tile's last row
    return max(0, held - (n - 1 - min(q, n - 1)));
  }
  // a tile that sees nothing still has its rows written
  __device__ __forceinline__ int steps() const { return max(1, (int)(((unsigned)sees() + kKeys - 1) / kKeys)); }
  __device__ __forceinline__ long long head_steps() {  // of all tiles of one head; ends at tile 0
    long long sum = 0;
    for (first_tile(); t < tiles; next_tile()) sum += steps();
    first_tile();
    return sum;
  }
  __device__ __forceinline__ void next_unit(const Cache4AttnArgs& a) {
    next_tile();
    if (t < tiles) return;
    first_tile();
    if (++h < a.Hkv) return;
    h = 0;
    do {
      r++;
      if (r >= a.R) return;
      request(a, r);
    } while (tiles == 0);
  }
  __device__ __forceinline__ int rows() const { return min(2 * kRows, n * group - t * 2 * kRows); }
};

// A warp's place on the line. In shared memory: inside a unit its registers are needed elsewhere.
struct Place {
  Walk wk;
  int s_begin;
  long long left, at, chunk;   // steps to go; where the unit begins on the line; steps of a CTA

  // steps of this unit that are the CTA's own
  __device__ __forceinline__ int steps() const { return (int)min((long long)wk.steps() - s_begin, left); }
  __device__ __forceinline__ void next(const Cache4AttnArgs& a, int lane) {
    __syncwarp();
    if (lane == 0) {
      const int n = steps();
      at += wk.steps();
      left -= n;
      s_begin = 0;
      wk.next_unit(a);
    }
    __syncwarp();
  }
};

struct Shared {
  uint64_t q_full[2], q_empty[2], kv_full[2], kv_empty[2];
  uint64_t s_full[2], p_full[2], o_final[2], drain;
  AbortState abort;
  uint32_t tmem;
  float factor[2][2][kRows];   // scores' factor of each row, of even and odd units of a tile
  Place place[kThreads / 32];
  long long scan[kThreads / 32];
  Walk found;                // the unit that the run begins in, and its place on the line
  long long line0;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 1024 + code, and 64 + code, of a word's codes 0 and 4, and 1 and 5, in fp16.
__device__ __forceinline__ uint32_t codes04(uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(r) : "r"(x), "r"(0x64006400u));
  return r;
}
__device__ __forceinline__ uint32_t codes15(uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(r) : "r"(x), "r"(0x54005400u));
  return r;
}
__device__ __forceinline__ uint32_t value2(uint32_t code, uint32_t offset, __half2 scale, __half2 low) {
  const __half2 c = __hsub2(*reinterpret_cast<__half2*>(&code), *reinterpret_cast<__half2*>(&offset));
  const __half2 v = __hfma2(c, scale, low);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Eight values of a word, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 values8(uint32_t x, __half2 scale, __half2 low) {
  const uint32_t y = x >> 8;
  return make_uint4(value2(codes04(x), 0x64006400u, scale, low), value2(codes15(x), 0x54005400u, scale, low),
                    value2(codes04(y), 0x64006400u, scale, low), value2(codes15(y), 0x54005400u, scale, low));
}
__device__ __forceinline__ __half2 twice_lo(uint32_t x) { return __low2half2(*reinterpret_cast<__half2*>(&x)); }
__device__ __forceinline__ __half2 twice_hi(uint32_t x) { return __high2half2(*reinterpret_cast<__half2*>(&x)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
template <int N>
__device__ __forceinline__ void ld_shared(uint32_t at, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 1)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at));
}

// kind::f16 with fp16 operands and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ------------------------------------------------------------------ softmax

// Waits for this thread's TMEM loads; x, one of their destinations, is not read before.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]),
                 "+r"(x[15]), "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]),
                 "+r"(x[22]), "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]),
                 "+r"(x[29]), "+r"(x[30]), "+r"(x[31])
               :
               : "memory");
}
// 32 scores of a row; those of keys from `seen` on (counted from the first) become -inf.
__device__ __forceinline__ void hide32(bool cut, int seen, uint32_t (&x)[32]) {
  if (cut)
#pragma unroll
    for (int c = 0; c < 32; c++) x[c] = c < seen ? x[c] : 0xff800000u;
}
// P = exp2(S * factor + shift) of 32 scores as 16 fp16 pairs; their sum is added to acc. kRound: the product is rounded
// first, as the maximum's was.
template <bool kRound>
__device__ __forceinline__ void p32(const uint32_t (&x)[32], float factor, float shift, uint32_t* pk, uint64_t& acc) {
  const uint64_t f2 = f2pack(factor, factor), s2 = f2pack(shift, shift);
#pragma unroll
  for (int c = 0; c < 16; c++) {
    float a0, a1;
    const float s0 = __uint_as_float(x[2 * c]), s1 = __uint_as_float(x[2 * c + 1]);
    if (kRound) {  // (by intrinsics that are never made one multiply-add)
      a0 = __fadd_rn(__fmul_rn(s0, factor), shift);
      a1 = __fadd_rn(__fmul_rn(s1, factor), shift);
    } else {
      f2unpack(ffma2(f2pack(s0, s1), f2, s2), a0, a1);
    }
    const float p0 = ex2(a0), p1 = ex2(a1);
    acc = fadd2(acc, f2pack(p0, p1));
    pk[c] = pack_half2(p0, p1);
  }
}
__device__ __forceinline__ float both(uint64_t acc) {
  float r0, r1;
  f2unpack(acc, r0, r1);
  return r0 + r1;
}
// Brings 64 P that were written to a maximum that moved, by an exact power of two.
__device__ __forceinline__ void scale_p64(uint32_t tP, float f) {
  uint32_t x[32];
  tmem_ld32(tP, x);
  tmem_wait_ld32(x);
#pragma unroll
  for (int c = 0; c < 32; c++) {
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[c]));
    x[c] = pack_half2(y.x * f, y.y * f);
  }
  tmem_st32(tP, x);
}
// 2^k for an integral k <= 0 (k = -inf gives 0), exact.
__device__ __forceinline__ float exp2_int(float k) {
  return k < -126.f ? 0.f : __int_as_float((static_cast<int>(k) + 127) << 23);
}

// The row's P where the running maximum m does not serve: none yet, or scores far above it. The
// first `done` of the two halves of 64 have their P already (sum rs). Takes the maximum of the others,
// moves m to an integer kBelow under it, and writes P. Returns what the older sums have to be
// multiplied by. Warp-collective; out of the common path, it reads S twice.
__device__ __forceinline__ float p_anew(uint32_t tS, int done, bool cut, int seen, float factor, float& m, float& rs) {
  float top = -INFINITY;
  for (int c = 2 * done; c < 4; c++) {
    uint32_t x[32];
    tmem_ld32(tS + c * 32, x);
    tmem_wait_ld32(x);
    hide32(cut, seen - c * 32, x);
#pragma unroll
    for (int e = 0; e < 32; e += 2) top = fmax3(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
  }
  top = __fmul_rn(top, factor);
  // (their difference is exact where m + kGrow would round)
  const float mnew = top - m > kGrow ? ceilf(top) - (fabsf(top) < kLarge ? kBelow : 0.f) : m;
  const float alpha = mnew == m ? 1.f : exp2_int(m - mnew);   // (-inf - -inf)
  if (done == 1) {
    scale_p64(tS, alpha);
    rs *= alpha;
  }
  uint64_t acc = f2pack(0.f, 0.f);
  for (int h = done; h < 2; h++) {
    uint32_t x[32], pk[32];
#pragma unroll
    for (int c = 0; c < 2; c++) {
      tmem_ld32(tS + h * 64 + c * 32, x);
      tmem_wait_ld32(x);
      hide32(cut, seen - h * 64 - c * 32, x);
      // a row that has seen no key yet: its scores are all -inf
      p32<true>(x, factor, mnew == -INFINITY ? 0.f : -mnew, pk + 16 * c, acc);
    }
    tmem_st32(tS + h * 64, pk);
  }
  rs += both(acc);
  m = mnew;
  return alpha;
}

// ------------------------------------------------------------------ copies and dequantisation

// What a dequantising warp needs of a tile of 128 keys: its own sixteen tokens, and at a unit's first
// tile the unit's rows.
struct Tile {
  const uint8_t* src;     // their sub-block; null: nothing is copied (no key, or a page outside the cache)
  int keys;               // how many of them are keys of the request
  bool first;
  int row0, h, t, rows;
};

// Query rows of a tile of 128 in fp16. A power of two a row brings its largest channel to 2^8 .. 2^9
// (bf16's bits then fit, but for what is below 2^-29 of that channel); it returns in the scores'
// factor. The scale's sign goes with the row.
template <int D>
struct QueryRows {
  static constexpr int kLanes = D / 8, kPerWarp = 32 / kLanes;                      // lanes a row, rows a warp
  static constexpr int kMine = (kRows + kFillWarps * kPerWarp - 1) / (kFillWarps * kPerWarp);  // rows a lane
  uint4 x[kMine];
  __device__ __forceinline__ int row(int b) const {
    return (b * kFillWarps + (threadIdx.x >> 5) - kFill0) * kPerWarp + (threadIdx.x & 31) / kLanes;
  }
  __device__ __forceinline__ void load(const Cache4AttnArgs& a, const Tile& u, int t) {
    const int ch = threadIdx.x % kLanes, rows = min(kRows, u.rows - t * kRows), group = a.Hq / a.Hkv;
#pragma unroll
    for (int b = 0; b < kMine; b++) {
      x[b] = make_uint4(0u, 0u, 0u, 0u);
      if (row(b) < rows) {
        const int full = u.t * 2 * kRows + t * kRows + row(b), i = full / group;
        x[b] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (u.row0 + i) * a.qs[0] +
                                               (u.h * group + full - i * group) * a.qs[1] + 8 * ch);
      }
    }
  }
  __device__ __forceinline__ void store(const Cache4AttnArgs& a, uint32_t dst, float* factor) const {
    const int ch = threadIdx.x % kLanes;
#pragma unroll
    for (int b = 0; b < kMine; b++) {
      const int r = row(b);
      const uint32_t y[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
      float f[8], big = 0.f;
#pragma unroll
      for (int z = 0; z < 4; z++) {
        f[2 * z] = __uint_as_float(y[z] << 16);
        f[2 * z + 1] = __uint_as_float(y[z] & 0xffff0000u);
        big = fmax3(big, fabsf(f[2 * z]), fabsf(f[2 * z + 1]));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      const int ex = max((int)(__float_as_uint(big) >> 23), 9);
      float down = __uint_as_float((uint32_t)(262 - ex) << 23);
      down = a.scale < 0.f ? -down : a.scale == 0.f ? 0.f : down;
      // A row with an infinity has no softmax. Its scores may all be -inf, which marks hidden keys: NaN instead.
      if (big == INFINITY) down = NAN;
      if (r < kRows) {
        st_shared16(dst + (ch >> 3) * Layout<D>::half + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                    make_uint4(pack_half2(f[0] * down, f[4] * down), pack_half2(f[1] * down, f[5] * down),
                               pack_half2(f[2] * down, f[6] * down), pack_half2(f[3] * down, f[7] * down)));
        if (ch == 0)  // never 0 or infinite: a hidden score times it stays -inf, and one of 0 stays 0
          factor[r] = fminf(fmaxf(__uint_as_float((uint32_t)(ex - 8) << 23) * fabsf(a.scale) * 1.4426950408889634f, 1.2e-38f), 3.4e38f);
      }
    }
  }
};

// Warp w takes tokens 16 w .. 16 w + 15 of every tile of the run. Phase g writes K of tile g and V of
// tile g - 1: those buffers come free, and are needed, together.
template <int D>
__device__ __forceinline__ void fill(const Cache4AttnArgs& a, Shared& sh, uint32_t smem, Place& place,
                                     const Abort ab) {
  using L = Layout<D>;
  constexpr int NG = D / 32;
  const int w = (threadIdx.x >> 5) - kFill0, lane = threadIdx.x & 31;
  const int c = lane & 3, u8 = ((lane >> 2) & 1) * 4 + (lane >> 3), v8 = c4::v_row(u8);
  const uint32_t raw_k = smem + L::ring + w * 2 * L::piece, raw_v = raw_k + L::piece;
  // where this lane's 16-byte chunks of token u8 lie in an operand: groups 0, 1 (and 2, 3 in the next half)
  const uint32_t at0 = w * 16 * 128 + u8 * 128 + ((c ^ u8) << 4), at1 = at0 ^ 64;

  // the run's tiles in order, one ahead of the copies
  int e = 0, n = 0;                 // tile of the unit, and the unit's tiles
  int pages = 0, pages_next = 0;    // this warp's page numbers of 32 tiles, a lane each, and of the next 32
  auto page_of = [&](int tile) {
    const unsigned k0 = (unsigned)(place.s_begin + tile) * kKeys + w * 16;
    return k0 < (unsigned)place.wk.held ? a.table[place.wk.r * a.table_stride + (k0 >> a.page_shift)] : -1;
  };
  auto next_tile = [&](Tile& x) {
    if (e == n) {
      if (n > 0) place.next(a, lane);
      e = n = 0;
      if (place.left <= 0) return false;
      n = place.steps();
      pages_next = page_of(lane);
    }
    if ((e & 31) == 0) {
      pages = pages_next;
      pages_next = page_of(e + 32 + lane);
    }
    const int page = __shfl_sync(0xffffffffu, pages, e & 31);
    const unsigned k0 = (unsigned)(place.s_begin + e) * kKeys + w * 16;
    x.keys = k0 < (unsigned)place.wk.held ? (int)min((unsigned)place.wk.held - k0, 16u) : 0;
    x.src = x.keys > 0 && (unsigned)page < (unsigned)a.n_pages
                ? a.cache + ((((size_t)page * a.Hkv + place.wk.h) << (a.page_shift - 4)) +
                             ((k0 & ((1u << a.page_shift) - 1)) >> 4)) * c4::sub_bytes(D)
                : nullptr;
    x.first = e == 0;
    if (e == 0) {
      x.row0 = place.wk.row0;
      x.h = place.wk.h;
      x.t = place.wk.t;
      x.rows = place.wk.rows();
    }
    e++;
    return true;
  };
  auto copy = [&](const uint8_t* src, uint32_t dst) {
    if (src)
#pragma unroll
      for (int at = 0; at < (int)L::piece; at += 512)
        if (at + 512 <= (int)L::piece || at + lane * 16 < (int)L::piece)
          cp_async16(dst + at + lane * 16, src + at + lane * 16);
  };

  Tile next, cur, prev;
  bool has_next = next_tile(next), has_cur = false, has_prev = false, ok = true;
  if (has_next) copy(next.src, raw_k);
  cp_async_commit();
  int units[2] = {0, 0};            // units so far that use rows of tile A, tile B
  int g = 0;
  for (;; g++) {
    has_prev = has_cur;
    has_cur = has_next;
    if (!has_prev && !has_cur) break;
    prev = cur;
    cur = next;
    cp_async_wait_all();
    __syncwarp();  // the wait is for this lane's copies; a vote would not order the others' before the reads below
    uint32_t kx[2][NG], sc[2][NG / 2], lo[2][NG / 2], vx[2][NG], pair[2][NG];
#pragma unroll
    for (int it = 0; it < 2; it++) {
      ld_shared(raw_v + (v8 + 8 * it) * 16 * NG + ((2 * c) ^ c4::v_turn(v8, NG)) * 2 * NG, vx[it]);
      ld_shared(raw_v + (c4::vp_at(D) - c4::vc_at(D)) + (v8 + 8 * it) * 4 * NG, pair[it]);
      ld_shared(raw_k + (u8 + 8 * it) * 16 * NG + c * 4 * NG, kx[it]);
      ld_shared(raw_k + c4::ks_at(D) + (u8 + 8 * it) * 2 * NG, sc[it]);
      ld_shared(raw_k + c4::km_at(D) + (u8 + 8 * it) * 2 * NG, lo[it]);
    }
    __syncwarp();
    has_next = has_cur && next_tile(next);
    if (has_next) copy(next.src, raw_k);
    if (has_cur && cur.src) copy(cur.src + c4::vc_at(D), raw_v);
    cp_async_commit();
    ok = __all_sync(0xffffffffu, mbar_wait<2>(smem_addr(&sh.kv_empty[g & 1]), ((g >> 1) & 1) ^ 1, ab));
    if (!ok) break;
    if (has_prev) {
      const uint32_t dst = smem + L::v + ((g - 1) & 1) * L::tile;
#pragma unroll
      for (int it = 0; it < 2; it++) {
        // what lies behind the last key, or was never copied, must not reach the sums: 0 * NaN
        const bool hide = !prev.src || u8 + 8 * it >= prev.keys;
#pragma unroll
        for (int j = 0; j < NG; j++) {
          const uint32_t word = __byte_perm(vx[it][j / 2], vx[it][NG / 2 + j / 2], (j & 1) ? 0x7632u : 0x5410u);
          const uint32_t pr = hide ? 0u : pair[it][j];
          st_shared16(dst + (j >> 1) * L::half + ((j & 1) ? at1 : at0) + it * 8 * 128,
                      values8(word, twice_lo(pr), twice_hi(pr)));
        }
      }
    }
    if (has_cur) {
      const uint32_t dst = smem + L::k + (g & 1) * L::tile;
#pragma unroll
      for (int it = 0; it < 2; it++)
#pragma unroll
        for (int j = 0; j < NG; j++) {
          // a page outside the cache: NaN, for every row that sees it
          const uint32_t s2 = cur.src ? sc[it][j / 2] : 0x7e007e00u, l2 = lo[it][j / 2];
          st_shared16(dst + (j >> 1) * L::half + ((j & 1) ? at1 : at0) + it * 8 * 128,
                      (j & 1) ? values8(kx[it][j], twice_hi(s2), twice_hi(l2))
                              : values8(kx[it][j], twice_lo(s2), twice_lo(l2)));
        }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.kv_full[g & 1]));
    if (has_cur && cur.first) {     // the unit's queries, after its first keys
#pragma unroll 1
      for (int t = 0; t < (cur.rows > kRows ? 2 : 1); t++) {
        const int k = t ? units[1] : units[0];
        QueryRows<D> qr;
        qr.load(a, cur, t);
        ok = __all_sync(0xffffffffu, mbar_wait<2>(smem_addr(&sh.q_empty[t]), (k & 1) ^ 1, ab));
        if (!ok) break;
        qr.store(a, smem + L::q + t * L::tile, sh.factor[k & 1][t]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[t]));
        t ? units[1]++ : units[0]++;
      }
      if (!ok) break;
    }
  }
  cp_async_wait_all();
}

// ------------------------------------------------------------------ the kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache4_tc_kernel(const __grid_constant__ Cache4AttnArgs a) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  Walk wk;
  wk.group = a.Hq / a.Hkv;
  wk.h = 0;

  // ---- this CTA's run of steps, and the unit that it starts in
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r_lo = min((int)threadIdx.x * per, a.R), r_hi = min(r_lo + per, a.R);
  long long mine = 0;
  for (int r = r_lo; r < r_hi; r++) {
    wk.request(a, r);
    mine += (long long)a.Hkv * wk.head_steps();
  }
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) sh.scan[warp] = before;
  const Abort ab{smem_addr(&sh.abort)};
  if (threadIdx.x == 0) {
    abort_state_init(sh.abort, a.status, kWaitLimitNs, 0);
    for (int s = 0; s < 2; s++) {
      mbar_init(smem_addr(&sh.q_full[s]), kFillWarps);
      // the last QK^T has read Q, and each softmax warp its factors
      mbar_init(smem_addr(&sh.q_empty[s]), 1 + 4);
      mbar_init(smem_addr(&sh.kv_full[s]), kFillWarps);
      mbar_init(smem_addr(&sh.kv_empty[s]), 1);
      mbar_init(smem_addr(&sh.s_full[s]), 1);
      mbar_init(smem_addr(&sh.p_full[s]), kRows);
      mbar_init(smem_addr(&sh.o_final[s]), 1);
    }
    mbar_init(smem_addr(&sh.drain), 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  long long total = 0;
  before -= mine;
  for (int i = 0; i < kThreads / 32; i++) {
    if (i < warp) before += sh.scan[i];
    total += sh.scan[i];
  }
  const long long chunk = max((total + gridDim.x - 1) / (long long)gridDim.x, (long long)a.min_chunk);
  const long long run0 = cta * chunk, run1 = min(run0 + chunk, total);
  if (run0 < total && before <= run0 && run0 < before + mine) {
    long long at = before;
    for (int r = r_lo; r < r_hi; r++) {
      wk.request(a, r);
      const long long one = wk.head_steps(), all = one * a.Hkv;
      if (run0 < at + all) {
        const int h = (int)((run0 - at) / one);
        at += h * one;
        while (run0 >= at + wk.steps()) {
          at += wk.steps();
          wk.next_tile();
        }
        wk.h = h;
        sh.found = wk;
        sh.line0 = at;
        break;
      }
      at += all;
    }
  }
  __syncthreads();
  long long left = max(0LL, run1 - run0);
  int s_begin = 0;
  if (left > 0) {
    wk = sh.found;
    s_begin = (int)(run0 - sh.line0);
  }

  Place& place = sh.place[warp];
  if (lane == 0) place = Place{wk, s_begin, left, sh.line0, chunk};
  __syncwarp();

  if (warp < kFill0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0) {
      // ---------------------------------------------------------------- MMA issuer
      const uint32_t idesc_qk = idesc_f16_f32(kRows, kKeys, false);
      const uint32_t idesc_pv = idesc_f16_f32(kRows, D, true);
      const uint64_t dQ = smem_desc_sw128(smem + L::q, 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem + L::k, 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem + L::v, L::half, 1024);
      constexpr uint32_t kTileDesc = L::tile >> 4;
      // Steps run on across units: a unit's last PVs go out in the next one's first step, so that
      // its softmax and its output run under the next one's first MMAs.
      int g = 0;                              // key tiles so far
      int units0 = 0, units1 = 0, p0 = 0, p1 = 0;   // units and p_full phases so far, of tile A and B
      int n = 0, j = 0;                       // steps of the unit, and the next one
      bool two = false, pv = false, pv_two = false, pv_on = false, pv_last = false;  // pv: of the last step
      bool ok = true;
      while (true) {
        const bool flush = place.left <= 0;
        if (flush && !pv) break;
        if (!flush && j == 0) {
          n = place.steps();
          two = place.wk.rows() > kRows;
        }
        const int gp = g - 1;
        ok = mbar_wait(smem_addr(&sh.kv_full[g & 1]), (g >> 1) & 1, ab);
        const uint64_t dKj = dK + (uint64_t)((g & 1) * kTileDesc), dVj = dV + (uint64_t)((gp & 1) * kTileDesc);
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * D;
          if (pv && (t == 0 || pv_two)) {
            ok = ok && mbar_wait(smem_addr(&sh.p_full[t]), (t ? p1 : p0) & 1, ab);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; kk++)
              mma_ts_elect(tO, tS + (kk >> 2) * 64 + (kk & 3) * 8, dVj + (uint64_t)(kk * (2048 >> 4)), idesc_pv,
                           kk ? 1u : (uint32_t)pv_on);
            t ? p1++ : p0++;
            if (pv_last) mma_commit_elect(smem_addr(&sh.o_final[t]));
          }
          if (!flush && (t == 0 || two)) {
            if (j == 0) ok = ok && mbar_wait(smem_addr(&sh.q_full[t]), (t ? units1 : units0) & 1, ab);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dQt = dQ + (uint64_t)(t * kTileDesc);
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++) {
              const uint64_t off = (uint64_t)(((kk >> 2) * L::half + (kk & 3) * 32) >> 4);
              mma_ss_elect(tS, dQt + off, dKj + off, idesc_qk, kk > 0);
            }
            mma_commit_elect(smem_addr(&sh.s_full[t]));
            if (j == n - 1) {
              mma_commit_elect(smem_addr(&sh.q_empty[t]));
              t ? units1++ : units0++;
            }
          }
        }
        if (!ok || flush) break;
        mma_commit_elect(smem_addr(&sh.kv_empty[g & 1]));
        pv = true;
        pv_two = two;
        pv_on = j > 0;
        pv_last = j == n - 1;
        g++;
        if (++j == n) {
          j = 0;
          place.next(a, lane);
        }
      }
      mma_commit_elect(smem_addr(&sh.drain));
      mbar_wait_drain(smem_addr(&sh.drain), 0, a.status, kWaitLimitNs);
      __syncwarp();
    }
  } else if (warp < kSoft0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFill));
    fill<D>(a, sh, smem, place, ab);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------------ softmax and O
    const int t = (warp - kSoft0) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + 256 + t * D;
    const bool scribe = threadIdx.x == 32 * kSoft0;   // writes the CTA's entry of the join list
    if (scribe) a.joins[2 * cta] = make_int4(0, 0, 0, 0);   // none, so far
    uint32_t scnt = 0;
    int unit = 0;
    while (place.left > 0) {
      int n, seen = 0;
      const bool used = t == 0 || place.wk.rows() > kRows;
      {
        const Walk wk = place.wk;
        const int steps = wk.steps(), s_begin = place.s_begin, rows = wk.rows();
        n = place.steps();
        if (scribe && s_begin == 0 && n < steps) {
          a.joins[2 * cta] = make_int4((int)((place.at + steps - 1) / place.chunk), rows, wk.t, wk.row0);
          a.joins[2 * cta + 1] = make_int4(wk.h, 0, 0, 0);
        }
        const int full = wk.t * 2 * kRows + t * kRows + row;
        const bool live = t * kRows + row < rows;
        // keys that the row sees, counted from the unit's first
        seen = (live ? max(0, wk.held - (wk.n - 1 - full / wk.group)) : wk.sees()) - s_begin * kKeys;
      }
      if (used) {
        float m = -INFINITY, l = 0.f;
        bool ok = __all_sync(0xffffffffu, mbar_wait<1>(smem_addr(&sh.q_full[t]), unit & 1, ab));
        if (!ok) break;
        const float factor = sh.factor[unit & 1][t][row];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_empty[t]));
        for (int j = 0; j < n; j++, scnt++, seen -= kKeys) {
          ok = __all_sync(0xffffffffu, mbar_wait<1>(smem_addr(&sh.s_full[t]), scnt & 1, ab));
          if (!ok) break;
          tc_fence_after();
          const bool cut = __any_sync(0xffffffffu, seen < kKeys);
          float rs = 0.f, alpha = 1.f;
          // The common case: every row of the warp has a maximum m (of ordinary size), and P with it does not
          // overflow, which the sum of P shows: no maximum is taken. P goes over the first 32 columns of its half of S.
          int done = 0;
          if (__all_sync(0xffffffffu, fabsf(m) < kLarge)) {
            uint32_t x[2][32], pk[32];
            tmem_ld32(tS, x[0]);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              uint64_t acc = f2pack(0.f, 0.f);
#pragma unroll
              for (int c = 0; c < 2; c++) {
                tmem_wait_ld32(x[c]);
                if (2 * h + c < 3) tmem_ld32(tS + (2 * h + c + 1) * 32, x[c ^ 1]);
                hide32(cut, seen - (2 * h + c) * 32, x[c]);
                p32<false>(x[c], factor, -m, pk + 16 * c, acc);
              }
              const float sum = both(acc);
              if (done != h || !__all_sync(0xffffffffu, sum <= kSumLimit)) continue;
              tmem_st32(tS + h * 64, pk);
              rs += sum;
              done++;
            }
          }
          if (done < 2) {
            tmem_wait_st();
            const float was = m;
            alpha = p_anew(tS, done, cut, seen, factor, m, rs);
            // PV of the previous tile has completed (S of this one landed after it)
            if (j > 0 && __any_sync(0xffffffffu, m != was)) {
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ch++) {
                uint32_t o[32];
                tmem_ld32(tO + ch * 32, o);
                tmem_wait_ld32(o);
#pragma unroll
                for (int c = 0; c < 32; c++) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                tmem_st32(tO + ch * 32, o);
              }
            }
          }
          l = l * alpha + rs;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_addr(&sh.p_full[t]));
        }
        ok = ok && mbar_wait<1>(smem_addr(&sh.o_final[t]), unit & 1, ab);
        unit++;
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();

        // ---- O, or this CTA's part of it
        const Walk wk = place.wk;
        const bool starts = place.s_begin == 0, whole = starts && n == wk.steps();
        const int full = wk.t * 2 * kRows + t * kRows + row;
        const bool live = t * kRows + row < wk.rows();
        const int i = live ? full / wk.group : 0;
        const int hq = wk.h * wk.group + (live ? full - i * wk.group : 0);
        const float inv = l == 0.f ? 0.f : whole ? 1.f / l : 1.f;
        const int part = 2 * cta + (starts ? 1 : 0);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + ((size_t)(wk.row0 + i) * a.Hq + hq) * D;
        float* dst_part = a.part_o + ((size_t)part * 2 * kRows + t * kRows + row) * D;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ch++) {
          uint32_t o[32];
          tmem_ld32(tO + ch * 32, o);
          tmem_wait_ld32(o);
          if (live) {
#pragma unroll
            for (int e = 0; e < 4; e++) {           // eight channels, in the order 0 4 1 5 2 6 3 7
              float f[8];
#pragma unroll
              for (int z = 0; z < 8; z++) f[z] = __uint_as_float(o[8 * e + (z & 3) * 2 + (z >> 2)]) * inv;
              if (whole) {
                *reinterpret_cast<uint4*>(dst + ch * 32 + 8 * e) =
                    make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                               pack_bf16x2(f[6], f[7]));
              } else {
                *reinterpret_cast<float4*>(dst_part + ch * 32 + 8 * e) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(dst_part + ch * 32 + 8 * e + 4) = make_float4(f[4], f[5], f[6], f[7]);
              }
            }
          }
        }
        tc_fence_before();
        if (live) {
          if (whole) {
            if (a.lse)
              a.lse[(size_t)hq * a.T + wk.row0 + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
          } else {
            float* ml = a.part_ml + (size_t)part * 4 * kRows + t * kRows + row;
            ml[0] = m;
            ml[2 * kRows] = l;
          }
        }
      }
      place.next(a, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the tile that CTA blockIdx.x of the first launch started and did not end.
// Eight threads a row, 32 rows a block.
template <int D>
__global__ void __launch_bounds__(256) cache4_tc_join_kernel(const __grid_constant__ Cache4AttnArgs a) {
  const int first = blockIdx.x;
  const int4 j0 = a.joins[2 * first], j1 = a.joins[2 * first + 1];
  const int last = j0.x, rows = j0.y, group = a.Hq / a.Hkv;
  const int row = blockIdx.y * 32 + (threadIdx.x >> 3), col = (threadIdx.x & 7) * 4;  // and every 32 more
  if (row >= rows) return;  // no tile: rows is 0
  const int full = j0.z * 2 * kRows + row, i = full / group, hq = j1.x * group + full - i * group;
  float M = -INFINITY, Ls = 0.f;
  for (int p = first; p <= last; p++) {
    const float* ml = a.part_ml + (size_t)(2 * p + (p == first)) * 4 * kRows + row;
    M = fmaxf(M, ml[0]);
  }
  const float top = M == -INFINITY ? 0.f : M;
  float sum[D / 8] = {};
#pragma unroll 2
  for (int p = first; p <= last; p++) {
    const int id = 2 * p + (p == first);
    const float* ml = a.part_ml + (size_t)id * 4 * kRows + row;
    const float f = ex2(ml[0] - top);
    Ls = fmaf(ml[2 * kRows], f, Ls);
    const float4* src = reinterpret_cast<const float4*>(a.part_o + ((size_t)id * 2 * kRows + row) * D + col);
#pragma unroll
    for (int e = 0; e < D / 32; e++) {
      const float4 y = src[8 * e];
      sum[4 * e] = fmaf(y.x, f, sum[4 * e]);
      sum[4 * e + 1] = fmaf(y.y, f, sum[4 * e + 1]);
      sum[4 * e + 2] = fmaf(y.z, f, sum[4 * e + 2]);
      sum[4 * e + 3] = fmaf(y.w, f, sum[4 * e + 3]);
    }
  }
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + ((size_t)(j0.w + i) * a.Hq + hq) * D + col;
#pragma unroll
  for (int e = 0; e < D / 32; e++)
    *reinterpret_cast<uint2*>(dst + 32 * e) =
        make_uint2(pack_bf16x2(sum[4 * e] * inv, sum[4 * e + 1] * inv), pack_bf16x2(sum[4 * e + 2] * inv, sum[4 * e + 3] * inv));
  if (a.lse && col == 0)
    a.lse[(size_t)hq * a.T + j0.w + i] = Ls == 0.f ? -INFINITY : (top + log2f(Ls)) * 0.6931471805599453f;
}

template <int D>
cudaError_t go(Cache4AttnArgs a, cudaStream_t st) {
  auto kernel = cache4_tc_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::bytes);
  if (e != cudaSuccess) return e;
  // setmaxnreg.inc waits until the registers it asks for are free: refuse to launch unless the split
  // fits what the launch hands out
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kernel))) return e;
  if (kRegsIssue + 2 * kRegsFill + 2 * kRegsSoftmax > 5 * fa.numRegs) return cudaErrorInvalidConfiguration;
  kernel<<<kCache4TcCtas, kThreads, Layout<D>::bytes, st>>>(a);
  if ((e = cudaGetLastError())) return e;
  cache4_tc_join_kernel<D><<<dim3(kCache4TcCtas, 2 * kRows / 32), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache4_tc(Cache4AttnArgs a, cudaStream_t st) {
  a.min_chunk = 4;
  return a.d == 64 ? go<64>(a, st) : go<128>(a, st);
}

}  // namespace s2
