// Attention over the 4-bit cache for bf16 queries, on the warps' tensor instructions.
//
// A step of decoding reads every stored key and value once and does little else, so the
// kernel is built around that read: 5/8 byte a value from HBM, turned into tensor operands in
// registers. A tile holds up to 8 NT query rows of one kv head (the heads that share it, times the
// request's tokens). Keys are the MMA's rows: S^T = K Q^T with K's codes as the A operand (16
// tokens by 16 channels) and the queries as B, so that 8 rows fill an MMA; the scores' 8 x 8
// blocks are transposed in registers (movmatrix) into the B operand of O^T = V^T P^T. The tcgen05
// instructions want at least 64 rows and operands in shared memory, which a dozen query rows
// cannot use and which would send each dequantised value through shared memory once more.
//
// k codes become fp16 operands by one logic operation for two: a code in the low bits of an fp16
// is the subnormal code 2^-24, in the next four bits 16 times that, which is taken out of the
// query's half of those channels; the 2^-24 goes into the scores' factor. A group's
// products with the codes are exact, its sum is fp32; its scale is applied to the sum, the
// minima go through one more MMA against the queries' sums over each group (split in two
// fp16 parts, which carry 22 bits). A query row is first scaled by a power of two so that fp16
// holds it (bf16 has fewer bits; what is lost is below 2^-29 of the row's largest channel);
// the power returns in the scores' factor.
// v codes become values minimum + scale * code in fp16, half a step (2^-11) off, and so do the
// probabilities: both well below the output's bf16. The probabilities are multiplied by 2^15 first, so that the
// largest lie near the top of fp16, those of 2^-29 still have all their bits and only those below 2^-40 are dropped: many
// small ones may be the whole output, where the largest ones' values are zero. (As a smaller maximum, without the products,
// the 15 would be lost in the rounding of scores beyond 2^24.) Maxima, sums and accumulators are fp32.
//
// Work is steps of 32 keys of a (request, kv head, tile). All steps of the call lie on one line
// and each CTA takes an equal run of them, whatever the requests' lengths, or, of short calls, one
// equal part of one tile; its four warps take every fourth step, each with its own ring of cp.async
// copies, and meet only at the end of a tile. A tile that several CTAs share is joined by the last of
// them to arrive, in the order of the runs, so that the bits do not depend on timing.
//
// Measured (B200; from one GPU to another times differ by 6%): 102400 tokens, 32 heads on 32 of 128: 119 to 126 us, 524 MB,
// 4.2 to 4.4 TB/s; 24 requests of up to 32768, 64 on 8 of 128: 151 to 162 us, 653 MB; 13 requests of up to 6001, 5 tokens,
// 32 on 8 of 64: 29 us, 29 MB. No unit is full: of the first, DRAM gives 64% of the copy rate, the ALU pipe (logic and
// permutes, which take the codes out of their words) is 59% busy, issue slots 65%. With three warps a scheduler a warp that does not
// issue waits for the ALU pipe and for its own last result, a third each. The copies alone take 90 us of 119, the loop
// without v 92, without three quarters of k 105. Three CTAs an SM with 168 registers did better than four with 128
// (127 us); a maximum that is kept (123), shifts as multiplications (128) and e4m3 operands for k's codes (142) did worse.
// The third is short of work: 47% of the issue slots, waits for results, pages and the other warps at a tile's two ends.
#include <math.h>

#include <type_traits>

#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"
#include "sm100.cuh"

namespace s2 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kStep = 32;  // keys of a step
constexpr float kUp = 0x1p15f;  // of the probabilities as operands, and so of the accumulators
constexpr int kTries = 4, kCutChunk = 128;
__device__ constexpr int kMore[kTries] = {0, 2, 5, 10};  // steps

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// (x & mask) | 0x64006400: fp16 1024 with a code in its low bits, twice.
__device__ __forceinline__ uint32_t code_lo(uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(r) : "r"(x), "r"(0x64006400u));
  return r;
}
__device__ __forceinline__ uint32_t code_hi(uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(r) : "r"(x), "r"(0x64006400u));
  return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float half_lo(uint32_t x) { return __low2float(*reinterpret_cast<__half2*>(&x)); }
__device__ __forceinline__ float half_hi(uint32_t x) { return __high2float(*reinterpret_cast<__half2*>(&x)); }

// NG words from shared memory by the widest loads.
template <int NG>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[NG]) {
  if constexpr (NG == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (NG == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < NG; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  }
}

// What a tile needs of its queries, made once for all warps.
template <int NG, int NT>
struct Queries {
  uint4 frag[NT][NG][32];   // B operands: of a group's two k-steps
  uint2 sums[NT][32];       // B operand of the minima
  float factor[NT * 8];     // score factor, log2 domain
  int keys[NT * 8];         // keys that the row sees
};

// A request's rows and keys.
struct Request {
  int row0, n, held, tiles, steps;
};
__device__ __forceinline__ Request request(const Cache4AttnArgs& a, int r, int tile_rows) {
  Request q;
  const int begin = a.cu[r], end = a.cu[r + 1];
  q.row0 = begin;
  q.n = begin >= 0 && end > begin && end <= a.T ? end - begin : 0;
  const long long cap = (long long)a.max_pages << a.page_shift;
  q.held = (int)min((long long)max(a.lens[r], 0), cap);
  q.tiles = (int)(((long long)q.n * (a.Hq / a.Hkv) + tile_rows - 1) / tile_rows);
  q.steps = max(1, (q.held + kStep - 1) / kStep);  // a request without keys still has its rows written
  return q;
}

template <int NG, int NT, int ST>
struct Smem {
  static constexpr int d = 32 * NG, step_bytes = 2 * c4::sub_bytes(d);
  union {
    uint8_t ring[kWarps][ST][step_bytes];
    float o[kWarps][8][d];
  };
  float m[kWarps][NT * 8], l[kWarps][NT * 8];
  Queries<NG, NT> q;
  long long scan[kWarps];
  int tries[kWarps][kTries];
  long long find_base;
  int find_r, last;
};

template <int NG, int NT, int ST, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) cache4_attn_kernel(const __grid_constant__ Cache4AttnArgs a) {
  constexpr int d = 32 * NG, SUB = c4::sub_bytes(d), ROWS = 8 * NT;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<Smem<NG, NT, ST>*>(smem_raw);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int group = a.Hq / a.Hkv;

  // ---- this CTA's run of steps, and the request that it starts in. Up to 32 requests are a lane each,
  // in every warp for itself; more are spread over the threads, and the warps' sums meet in shared memory.
  // (One request needs no sums.)
  const bool alone = a.R <= 32, one = a.R == 1;
  const int per = alone ? 1 : (a.R + kThreads - 1) / kThreads;
  const int r_lo = one ? 0 : min((alone ? lane : (int)threadIdx.x) * per, a.R), r_hi = min(r_lo + per, a.R);
  auto upto = [&](auto x) {  // sum over the lanes up to this one
    if (one) return x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int cta = blockIdx.x, grid = gridDim.x;
  long long chunk = a.min_chunk, mine = 0, before = 0, total = 0;
  int more = -1, ctas = 0, my_parts = 0, parts_before = 0;
  // Cuts every tile into equal parts of at most chunk + kMore[k] steps, k = 0 .. N - 1, and takes the first k
  // whose parts fit the grid.
  auto cut = [&](auto tries) {
    constexpr int N = decltype(tries)::value, W = (N + 1) / 2;
    int parts[2 * W], sums[2 * W];
#pragma unroll
    for (int k = 0; k < 2 * W; k++) parts[k] = 0;
    for (int r = r_lo; r < r_hi; r++) {
      const Request q = request(a, r, ROWS);
      const long long units = (long long)a.Hkv * q.tiles;
#pragma unroll
      for (int k = 0; k < N; k++) {
        const unsigned len = (unsigned)chunk + kMore[k];
        parts[k] = (int)min(parts[k] + units * ((q.steps + len - 1) / len), (long long)kCache4MaxCtas + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < W; k++) {  // two sums in a word: 32 lanes of at most kCache4MaxCtas + 1
      static_assert(32 * (kCache4MaxCtas + 1) < 1 << 15, "");
      const int both = upto(parts[2 * k] | parts[2 * k + 1] << 16);
      sums[2 * k] = both & 0xffff;
      sums[2 * k + 1] = both >> 16;
    }
    if (!alone) {
      if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; k++) sm.tries[w][k] = sums[k];
      __syncthreads();
    }
#pragma unroll
    for (int k = N - 1; k >= 0; k--) {
      int all = 0, earlier = 0;
      if (alone) {
        all = __shfl_sync(0xffffffffu, sums[k], 31);
      } else {
#pragma unroll
        for (int i = 0; i < kWarps; i++) {
          if (i < w) earlier += sm.tries[i][k];
          all += sm.tries[i][k];
        }
      }
      if (all <= grid) {
        more = kMore[k];
        ctas = all;
        my_parts = parts[k];
        parts_before = earlier + sums[k] - parts[k];
      }
    }
  };
  // A grid with room for all parts of min_chunk steps that the table's width allows needs no more than that.
  if (a.roomy) cut(std::integral_constant<int, 1>{});
  if (more < 0) {
    for (int r = r_lo; r < r_hi; r++) {
      const Request q = request(a, r, ROWS);
      mine += (long long)a.Hkv * q.tiles * q.steps;
    }
    before = upto(mine);
    if (alone) {
      total = __shfl_sync(0xffffffffu, before, 31);
    } else {
      if (lane == 31) sm.scan[w] = before;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; i++) {
        if (i < w) before += sm.scan[i];
        total += sm.scan[i];
      }
    }
    before -= mine;
    chunk = max(total < (1LL << 31) - grid ? (long long)(((unsigned)total + grid - 1) / (unsigned)grid)
                                           : (total + grid - 1) / grid,
                (long long)a.min_chunk);
    // Equal runs of the line. Shorter ones end where tiles end, if a few steps more than that allow it (a
    // step is 0.4 us of a CTA): no CTA then visits two tiles, each with its queries, sums and join (5 us).
    // 3 requests of up to 5000 keys, 32 heads on 2 of 128: 21.8 us against 26.5; 8 of 4096, 64 on 8: 18.8
    // against 20.8; with 230 steps a CTA it is a loss.
    if (chunk <= kCutChunk) cut(std::integral_constant<int, kTries>{});
  }
  const long long run0 = cta * chunk;
  if (more >= 0 ? cta >= ctas : run0 >= total) return;
  int found = -1;
  long long at = more >= 0 ? parts_before : before;  // parts, or steps, of the requests before
  const long long goal = more >= 0 ? cta : run0, ahead = more >= 0 ? my_parts : mine;
  if (at <= goal && goal < at + ahead) {
    for (found = r_lo;; found++) {
      const Request q = request(a, found, ROWS);
      const int len = (int)chunk + more;
      const long long size = (long long)a.Hkv * q.tiles * (more >= 0 ? (q.steps + len - 1) / len : q.steps);
      if (goal < at + size) break;
      at += size;
    }
  }
  int r;
  if (alone) {
    const int who = __ffs(__ballot_sync(0xffffffffu, found >= 0)) - 1;
    r = __shfl_sync(0xffffffffu, found, who);
    at = __shfl_sync(0xffffffffu, at, who);
  } else {
    if (found >= 0) {
      sm.find_r = found;
      sm.find_base = at;
    }
    __syncthreads();
    r = sm.find_r;
    at = sm.find_base;
  }
  Request rq = request(a, r, ROWS);
  long long base, pos, run1;      // where request r's steps begin on the line; this CTA's run
  int part_of = 0, parts_of = 0;  // its part, of how many, of a tile that is cut into equal ones
  if (more >= 0) {
    const int len = (int)chunk + more;
    parts_of = (rq.steps + len - 1) / len;
    const int part = cta - (int)at, unit = part / parts_of;
    part_of = part - unit * parts_of;
    base = 0;
    const int equal = (rq.steps + parts_of - 1) / parts_of;  // at most len, so that none is empty
    pos = (long long)unit * rq.steps + part_of * equal;
    run1 = (long long)unit * rq.steps + min(rq.steps, (part_of + 1) * equal);
  } else {
    base = at;
    pos = run0;
    run1 = min(run0 + chunk, total);
  }
  while (pos < run1) {
    while (pos >= base + (long long)a.Hkv * rq.tiles * rq.steps) {
      base += (long long)a.Hkv * rq.tiles * rq.steps;
      rq = request(a, ++r, ROWS);
    }
    const long long into = pos - base;
    const int unit = into < (1LL << 31) ? (int)((unsigned)into / (unsigned)rq.steps) : (int)(into / rq.steps);
    const long long unit0 = base + (long long)unit * rq.steps;
    const int h = unit / rq.tiles, tile = unit - h * rq.tiles;
    const int s_begin = (int)(pos - unit0);
    const int s_end = (int)min((long long)rq.steps, run1 - unit0);
    const int rows = min(ROWS, rq.n * group - tile * ROWS);
    // keys of the tile's first and last row
    const int see_min = max(0, rq.held - (rq.n - 1 - tile * ROWS / group));
    const int see_max = max(0, rq.held - (rq.n - 1 - (tile * ROWS + rows - 1) / group));
    const int* table = a.table + r * a.table_stride;

    __syncthreads();  // the last tile's readers of sm are done

    // ---- this warp's steps: w, w + 4, ...; the first copies fly while the queries are prepared
    const int last = min(s_end, (see_max + kStep - 1) / kStep);
    uint8_t* ring = &sm.ring[w][0][0];
    const uint32_t ring_at = sm100::smem_addr(ring);
    int next = s_begin + w;          // step that is copied next
    int page0 = 0, page1 = 0;        // its pages (one each 16 keys)
    uint32_t bad = 0;                // two bits a ring slot: a page outside the cache
    auto load_pages = [&](int s) {
      if (s < last) {
        const int k0 = s * kStep;
        page0 = table[k0 >> a.page_shift];
        page1 = k0 + 16 < rq.held ? table[(k0 + 16) >> a.page_shift] : -1;
      }
    };
    auto issue = [&](int s, int slot) {
      bad &= ~(3u << (2 * slot));
      if (s < last) {
        const int k0 = s * kStep, in_page = (k0 & ((1 << a.page_shift) - 1)) >> 4;
        const bool ok0 = (unsigned)page0 < (unsigned)a.n_pages;
        const bool ok1 = (unsigned)page1 < (unsigned)a.n_pages;
        bad |= ((ok0 ? 0u : 1u) | (ok1 ? 0u : 2u)) << (2 * slot);
        const uint8_t* src0 = a.cache + ((((size_t)page0 * a.Hkv + h) << (a.page_shift - 4)) + in_page) * SUB + lane * 16;
        const uint8_t* src1 = a.cache + ((((size_t)page1 * a.Hkv + h) << (a.page_shift - 4)) +
                                         (a.page_shift == 4 ? 0 : in_page + 1)) * SUB + lane * 16;
        const uint32_t dst = ring_at + slot * (2 * SUB) + lane * 16;
        // a sub-block is FULL copies of 512 bytes, and the rest by the first lanes
        constexpr int FULL = SUB / 512, REST = SUB % 512 / 16;
        if (ok0) {
#pragma unroll
          for (int i = 0; i < FULL; i++) cp_async16(dst + i * 512, src0 + i * 512);
          if (REST && lane < REST) cp_async16(dst + FULL * 512, src0 + FULL * 512);
        }
        if (ok1) {
#pragma unroll
          for (int i = 0; i < FULL; i++) cp_async16(dst + SUB + i * 512, src1 + i * 512);
          if (REST && lane < REST) cp_async16(dst + SUB + FULL * 512, src1 + FULL * 512);
        }
      }
      cp_async_commit();
    };
    load_pages(next);
#pragma unroll
    for (int k = 0; k < ST; k++) {
      issue(next, k);
      next += kWarps;
      load_pages(next);
    }

    // ---- the tile's queries
    for (int nt = w; nt < NT; nt += kWarps) {
      const int row = tile * ROWS + nt * 8 + g;  // of this lane's quad
      const bool live = row < rq.n * group;
      const int i = live ? row / group : 0;
      float x[NG][8], big = 0.f;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                 (rq.row0 + i) * a.qs[0] + (h * group + (live ? row - i * group : 0)) * a.qs[1];
#pragma unroll
      for (int j = 0; j < NG; j++) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) raw = *reinterpret_cast<const uint4*>(src + 32 * j + 8 * c);
        const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
          x[j][2 * e] = __uint_as_float(v[e] << 16);
          x[j][2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
          big = fmaxf(big, fmaxf(fabsf(x[j][2 * e]), fabsf(x[j][2 * e + 1])));
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // a power of two that brings the largest channel to 2^8 .. 2^9 (a group's sum stays
      // below 2^14), from its exponent
      const int ex = max((int)(__float_as_uint(big) >> 23), 9);
      const float down = __uint_as_float((uint32_t)(262 - ex) << 23), up = __uint_as_float((uint32_t)(ex - 8) << 23);
      float part[NG];
#pragma unroll
      for (int j = 0; j < NG; j++) {
        part[j] = 0.f;
        __half y[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float xe = x[j][e] * down;
          y[e] = __float2half_rn((e & 1) ? xe * 0.0625f : xe);
          const float ye = __half2float(y[e]);
          part[j] += (e & 1) ? 16.f * ye : ye;
        }
        const __half2 f[4] = {__halves2half2(y[0], y[4]), __halves2half2(y[1], y[5]),
                              __halves2half2(y[2], y[6]), __halves2half2(y[3], y[7])};
        sm.q.frag[nt][j][lane] = *reinterpret_cast<const uint4*>(f);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) part[j] += __shfl_xor_sync(0xffffffffu, part[j], o);
      }
      // groups 2c, 2c + 1 of this row: high parts against the first eight k, low ones after
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < NG; j++) {
        if (j == 2 * c) s0 = part[j];
        if (j == 2 * c + 1) s1 = part[j];
      }
      const float h0 = __half2float(__float2half_rn(s0)), h1 = __half2float(__float2half_rn(s1));
      sm.q.sums[nt][lane] = make_uint2(pack_half2(h0, h1), pack_half2(s0 - h0, s1 - h1));
      if (c == 0) {
        // finite: a score of 0 times infinity would be NaN (queries of 2^115 and more)
        sm.q.factor[nt * 8 + g] = fminf(fmaxf(up * a.scale * (1.4426950408889634f * 0x1p24f), -3.4e38f), 3.4e38f);
        sm.q.keys[nt * 8 + g] = live ? max(0, rq.held - (rq.n - 1 - i)) : see_max;
      }
    }
    __syncthreads();

    uint4 qreg[NT == 1 ? NG : 1];
    if constexpr (NT == 1) {
#pragma unroll
      for (int j = 0; j < NG; j++) qreg[j] = sm.q.frag[0][j][lane];
    }

    float O[2 * NG][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * NG; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) O[i][nt][e] = 0.f;
    }

    int slot = 0;
    for (int s = s_begin + w; s < last; s += kWarps) {
      cp_async_wait<ST - 1>();
      __syncwarp();
      const uint8_t* stage = ring + slot * (2 * SUB);
      const uint32_t bad_here = (bad >> (2 * slot)) & 3u;
      const int k0 = s * kStep;

      // scores of 2 x 16 keys
      float S[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; mt++) {
        const uint8_t* sub = stage + mt * SUB;
        uint32_t kw[2][NG], sc[2][(NG + 1) / 2], mn[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int u = g + 8 * e;
          if constexpr (NG == 8) {
            uint32_t half[4];
            load_words<4>(sub + u * 128 + c * 32 + (u & 1) * 16, half);
#pragma unroll
            for (int i = 0; i < 4; i++) kw[e][i] = half[i];
            load_words<4>(sub + u * 128 + c * 32 + ((u & 1) ^ 1) * 16, half);
#pragma unroll
            for (int i = 0; i < 4; i++) kw[e][4 + i] = half[i];
          } else {
            load_words<NG>(sub + u * 16 * NG + c * 4 * NG, kw[e]);
          }
          load_words<NG / 2>(sub + c4::ks_at(d) + u * 2 * NG, sc[e]);
          mn[e] = 2 * c < NG ? *reinterpret_cast<const uint32_t*>(sub + c4::km_at(d) + u * 2 * NG + 4 * c) : 0u;
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          const uint2 z = sm.q.sums[nt][lane];
#pragma unroll
          for (int e = 0; e < 4; e++) S[mt][nt][e] = 0.f;
          mma16816(S[mt][nt], mn[0], mn[1], mn[0], mn[1], z.x, z.y);
#pragma unroll
          for (int e = 0; e < 4; e++) S[mt][nt][e] *= 0x1p-24f;
        }
#pragma unroll
        for (int j = 0; j < NG; j++) {
          const uint32_t x0 = kw[0][j], x1 = kw[1][j], y0 = x0 >> 8, y1 = x1 >> 8;
          constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
          const float s0 = (j & 1) ? half_hi(sc[0][j / 2]) : half_lo(sc[0][j / 2]);
          const float s1 = (j & 1) ? half_hi(sc[1][j / 2]) : half_lo(sc[1][j / 2]);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            const uint4 q = NT == 1 ? qreg[NT == 1 ? j : 0] : sm.q.frag[nt][j][lane];
            float C[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(C, x0 & lo, x1 & lo, x0 & hi, x1 & hi, q.x, q.y);
            mma16816(C, y0 & lo, y1 & lo, y0 & hi, y1 & hi, q.z, q.w);
            S[mt][nt][0] = fmaf(C[0], s0, S[mt][nt][0]);
            S[mt][nt][1] = fmaf(C[1], s0, S[mt][nt][1]);
            S[mt][nt][2] = fmaf(C[2], s1, S[mt][nt][2]);
            S[mt][nt][3] = fmaf(C[3], s1, S[mt][nt][3]);
          }
        }
      }

      // softmax, a running maximum and sum for each of this lane's two rows of a tile of eight
      const bool whole = k0 + kStep <= see_min && bad_here == 0;
      uint32_t P[2][NT][2];
      bool grew = false;
      float alpha[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        const float2 f = *reinterpret_cast<const float2*>(&sm.q.factor[nt * 8 + 2 * c]);
#pragma unroll
        for (int mt = 0; mt < 2; mt++) {
          S[mt][nt][0] *= f.x;
          S[mt][nt][1] *= f.y;
          S[mt][nt][2] *= f.x;
          S[mt][nt][3] *= f.y;
        }
        if (!whole) {
          const int2 see = *reinterpret_cast<const int2*>(&sm.q.keys[nt * 8 + 2 * c]);
#pragma unroll
          for (int mt = 0; mt < 2; mt++) {
            const int key = k0 + 16 * mt + g;
            const float other = (bad_here >> mt) & 1u ? NAN : 0.f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const bool seen = key + (e & 2 ? 8 : 0) < ((e & 1) ? see.y : see.x);
              S[mt][nt][e] = seen ? ((bad_here >> mt) & 1u ? other : S[mt][nt][e]) : -INFINITY;
            }
          }
        }
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float t = fmaxf(fmaxf(S[0][nt][e], S[0][nt][e + 2]), fmaxf(S[1][nt][e], S[1][nt][e + 2]));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          t = fmaxf(t, m[nt][e]);
          grew |= t > m[nt][e];
          top[e] = t == -INFINITY ? 0.f : t;
          alpha[nt][e] = ex2(m[nt][e] - top[e]);
          m[nt][e] = t;
        }
#pragma unroll
        for (int mt = 0; mt < 2; mt++) {
#pragma unroll
          for (int e = 0; e < 4; e++) S[mt][nt][e] = ex2(S[mt][nt][e] - top[e & 1]);
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float p0, p1;
            sm100::f2unpack(sm100::fmul2(sm100::f2pack(S[mt][nt][2 * e], S[mt][nt][2 * e + 1]), sm100::f2pack(kUp, kUp)), p0, p1);
            P[mt][nt][e] = transpose8(pack_half2(p0, p1));
          }
        }
#pragma unroll
        for (int e = 0; e < 2; e++)
          l[nt][e] = fmaf(l[nt][e], alpha[nt][e],
                          (S[0][nt][e] + S[0][nt][e + 2]) + (S[1][nt][e] + S[1][nt][e + 2]));
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < 2 * NG; i++)
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 4; e++) O[i][nt][e] *= alpha[nt][e & 1];
      }

      // values: lane (g, c) has four channels of each group of keys 2c, 2c + 1, 2c + 8, 2c + 9
      const bool tail = k0 + kStep > rq.held || bad_here != 0;
#pragma unroll
      for (int mt = 0; mt < 2; mt++) {
        const uint8_t* sub = stage + mt * SUB;
        uint32_t vw[4][(NG + 1) / 2], vp[4][NG];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int row = 4 * e + c;
          load_words<NG / 2>(sub + c4::vc_at(d) + row * 16 * NG + (g ^ c4::v_turn(c, NG)) * 2 * NG, vw[e]);
          load_words<NG>(sub + c4::vp_at(d) + row * 4 * NG, vp[e]);
          if (tail) {
            // what lies behind the last key, or was never copied, must not reach the sums: 0 * NaN
            const int key = k0 + 16 * mt + 2 * c + (e & 1) + (e & 2 ? 8 : 0);
            if (key >= rq.held || ((bad_here >> mt) & 1u))
#pragma unroll
              for (int j = 0; j < NG; j++) vp[e][j] = 0u;
          }
        }
#pragma unroll
        for (int j = 0; j < NG; j++) {
          const uint32_t pick = (j & 1) ? 0x7632u : 0x5410u;
          uint32_t A[2][4];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const uint32_t x = __byte_perm(vw[2 * e][j / 2], vw[2 * e + 1][j / 2], pick), y = x >> 8;
            const uint32_t scale = __byte_perm(vp[2 * e][j], vp[2 * e + 1][j], 0x5410u);
            const uint32_t low = __byte_perm(vp[2 * e][j], vp[2 * e + 1][j], 0x7632u);
            A[0][2 * e] = hfma2(hsub2(code_lo(x), 0x64006400u), scale, low);
            A[0][2 * e + 1] = hfma2(hfma2(code_hi(x), 0x2c002c00u, 0xd400d400u), scale, low);
            A[1][2 * e] = hfma2(hsub2(code_lo(y), 0x64006400u), scale, low);
            A[1][2 * e + 1] = hfma2(hfma2(code_hi(y), 0x2c002c00u, 0xd400d400u), scale, low);
          }
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            mma16816(O[2 * j][nt], A[0][0], A[0][1], A[0][2], A[0][3], P[mt][nt][0], P[mt][nt][1]);
            mma16816(O[2 * j + 1][nt], A[1][0], A[1][1], A[1][2], A[1][3], P[mt][nt][0], P[mt][nt][1]);
          }
        }
      }
      __syncwarp();  // the slot is read: it may be filled again
      issue(next, slot);
      next += kWarps;
      load_pages(next);
      slot = slot + 1 == ST ? 0 : slot + 1;
    }
    cp_async_wait<0>();

    // ---- the warps' parts
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          sm.l[w][nt * 8 + 2 * c + e] = x;
          sm.m[w][nt * 8 + 2 * c + e] = m[nt][e];
        }
      }
    const bool starts = s_begin == 0, ends = s_end == rq.steps;
    const int part = 2 * blockIdx.x + (starts ? 1 : 0);
    float* part_o = a.part_o + (size_t)part * kCache4PartFloats;
    float* part_ml = a.part_ml + (size_t)part * 2 * kCache4PartRows;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NG; j++)
#pragma unroll
        for (int e = 0; e < 2; e++)
          *reinterpret_cast<float4*>(&sm.o[w][2 * c + e][32 * j + 4 * g]) =
              make_float4(O[2 * j][nt][e], O[2 * j][nt][e + 2], O[2 * j + 1][nt][e], O[2 * j + 1][nt][e + 2]);
      __syncthreads();
      for (int x = threadIdx.x; x < 8 * d / 4; x += kThreads) {
        const int qi = x / (d / 4), col = (x - qi * (d / 4)) * 4, row = nt * 8 + qi;
        if (row >= rows) continue;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; i++) M = fmaxf(M, sm.m[i][row]);
        const float top = M == -INFINITY ? 0.f : M;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kWarps; i++) {
          const float f = ex2(sm.m[i][row] - top);
          const float4 y = *reinterpret_cast<const float4*>(&sm.o[i][qi][col]);
          L = fmaf(sm.l[i][row], f, L);
          sum.x = fmaf(y.x, f, sum.x);
          sum.y = fmaf(y.y, f, sum.y);
          sum.z = fmaf(y.z, f, sum.z);
          sum.w = fmaf(y.w, f, sum.w);
        }
        if (starts && ends) {
          const int full = tile * ROWS + row, i = full / group, hq = h * group + full - i * group;
          const float inv = L == 0.f ? 0.f : 1.f / (L * kUp);
          const uint2 out = make_uint2(sm100::pack_bf16x2(sum.x * inv, sum.y * inv),
                                       sm100::pack_bf16x2(sum.z * inv, sum.w * inv));
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) +
                                    ((size_t)(rq.row0 + i) * a.Hq + hq) * d + col) = out;
          if (a.lse && col == 0)
            a.lse[(size_t)hq * a.T + rq.row0 + i] = L == 0.f ? -INFINITY : (top + log2f(L)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float4*>(part_o + row * d + col) = sum;
          if (col == 0) {
            part_ml[row] = M;
            part_ml[kCache4PartRows + row] = L;
          }
        }
      }
    }

    // ---- a tile of several CTAs: the last to arrive joins the parts, in order
    if (!(starts && ends)) {
      const int first = parts_of ? cta - part_of : (int)(unit0 / chunk);
      const int final = parts_of ? first + parts_of - 1 : (int)((unit0 + rq.steps - 1) / chunk);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int was = (int)atomicAdd(a.counters + first, 1u);
        sm.last = was == final - first;
        if (sm.last) a.counters[first] = 0u;  // ready for the next call
      }
      __syncthreads();
      if (sm.last) {
        __threadfence();
        for (int x = threadIdx.x; x < rows * d / 4; x += kThreads) {
          const int row = x / (d / 4), col = (x - row * (d / 4)) * 4;
          float M = -INFINITY, L = 0.f;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int p = first; p <= final; p++) {
            const int id = 2 * p + (p == first ? 1 : 0);
            const float* ml = a.part_ml + (size_t)id * 2 * kCache4PartRows;
            const float mp = __ldcg(ml + row), lp = __ldcg(ml + kCache4PartRows + row);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(a.part_o + (size_t)id * kCache4PartFloats + row * d + col));
            const float Mn = fmaxf(M, mp), top = Mn == -INFINITY ? 0.f : Mn;
            const float f0 = ex2(M - top), f1 = ex2(mp - top);
            L = fmaf(L, f0, lp * f1);
            sum.x = fmaf(sum.x, f0, y.x * f1);
            sum.y = fmaf(sum.y, f0, y.y * f1);
            sum.z = fmaf(sum.z, f0, y.z * f1);
            sum.w = fmaf(sum.w, f0, y.w * f1);
            M = Mn;
          }
          const int full = tile * ROWS + row, i = full / group, hq = h * group + full - i * group;
          const float inv = L == 0.f ? 0.f : 1.f / (L * kUp), top = M == -INFINITY ? 0.f : M;
          const uint2 out = make_uint2(sm100::pack_bf16x2(sum.x * inv, sum.y * inv),
                                       sm100::pack_bf16x2(sum.z * inv, sum.w * inv));
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) +
                                    ((size_t)(rq.row0 + i) * a.Hq + hq) * d + col) = out;
          if (a.lse && col == 0)
            a.lse[(size_t)hq * a.T + rq.row0 + i] = L == 0.f ? -INFINITY : (top + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
    pos = unit0 + s_end;
  }
}

template <int NG, int NT, int ST, int MINB>
cudaError_t go(Cache4AttnArgs a, cudaStream_t st) {
  using S = Smem<NG, NT, ST>;
  static_assert(8 * NT * 32 * NG <= kCache4PartFloats && 8 * NT <= kCache4PartRows, "a part fits its place");
  auto kernel = cache4_attn_kernel<NG, NT, ST, MINB>;
  // set on every call: it is per device, and costs no synchronisation
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S));
  if (e != cudaSuccess) return e;
  // no more CTAs than the longest lengths the table allows can occupy, a run of min_chunk each
  const long long tiles = ((long long)a.max_new * (a.Hq / a.Hkv) + 8 * NT - 1) / (8 * NT);
  const long long steps = (((long long)a.max_pages << a.page_shift) + kStep - 1) / kStep;
  // (a double: max_new is only a hint and may be anything)
  const double parts = (double)a.R * a.Hkv * tiles * ((steps + a.min_chunk - 1) / a.min_chunk);
  a.roomy = parts <= 148 * MINB;
  const int ctas = a.roomy ? (int)parts : 148 * MINB;
  kernel<<<ctas, kThreads, sizeof(S), st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache4_attn(Cache4AttnArgs a, cudaStream_t st) {
  const long long rows = (long long)a.max_new * (a.Hq / a.Hkv);
  a.min_chunk = 2 * kWarps;
  if (a.d == 64) {
    if (rows <= 8) return go<2, 1, 4, 4>(a, st);
    if (rows <= 16) return go<2, 2, 4, 4>(a, st);
    if (rows <= 24) return go<2, 3, 4, 3>(a, st);
    return go<2, 4, 4, 3>(a, st);
  }
  if (a.d == 128) {
    if (rows <= 8) return go<4, 1, 2, 3>(a, st);
    if (rows <= 16) return go<4, 2, 3, 3>(a, st);
    if (rows <= 24) return go<4, 3, 3, 2>(a, st);
    return go<4, 4, 3, 2>(a, st);
  }
  if (rows <= 8) return go<8, 1, 2, 2>(a, st);
  return go<8, 2, 2, 2>(a, st);
}

}  // namespace s2
