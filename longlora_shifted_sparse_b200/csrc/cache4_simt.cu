// Attention over the 4-bit cache on the CUDA cores: every type and head dim, fp32 arithmetic.
//
// o = softmax(q k^T * scale) v for one token and up to four query heads of a kv head per CTA, over
// the keys up to the token's own place. Online softmax: each of four warps takes 32 keys at a time,
// a key a lane for the scores (a group's products with the codes are summed first, its scale and
// minimum applied once), then a few channels a lane for the values; the warps' (maximum, sum, output)
// are joined at the end. Keys the mask hides are never added, whatever their slots hold.
//
// Few rows are split over the keys, so that the calls that have them fill the GPU too: at least 128
// keys a CTA, the parts joined by the last of a row's CTAs to arrive, in order. Codes become floats
// through the mantissa, as conversions run at a quarter of the rate, and once for all heads of a CTA.
// Each warp copies its 32 keys, two sub-blocks, to shared memory before it reads them: its loads of codes
// are of four bytes, half a row and more apart.
// fp32 on a B200, us: one CTA a row; split; codes through the mantissa and heads together; keys copied:
// 100000 keys of one head of 64: 7796, 87, 53, 39; 1000 keys of 32 heads on 32 of 128: 86, 19, 19, 16;
// 4 requests of up to 4000 keys, 64 heads on 8 of 96: 347, 137, 79, 66. Bound by instructions: 68% of the
// issue slots and 13% of the memory's rate with 8 heads of 128 on 100000 keys (121 us).
#include <math.h>

#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"

namespace s2 {

constexpr int kSimtWarps = 4, kSimtSplits = 128;

// Code in bits 4 i (i < 4) of `word` as code * 16^i, exactly: it is the low end of 2^23's mantissa.
__device__ __forceinline__ float code_at(uint32_t word, int i) {
  return __uint_as_float((word & (15u << (4 * i))) | 0x4b000000u) - 8388608.f;
}

// A staged sub-block: its rows of k codes lie an odd number of 16-byte pieces apart, so that a warp's
// loads of one word of its rows meet four at a bank, the least that 16-byte copies allow.
__host__ __device__ constexpr int staged_bytes(int d) { return c4::sub_bytes(d) + 256; }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// H query heads of one kv head a CTA.
template <typename T, int H>
__global__ void __launch_bounds__(kSimtWarps * 32) cache4_attn_simt_kernel(
    const __grid_constant__ Cache4AttnArgs a) {
  __shared__ __align__(16) float q[H][256];
  __shared__ float qsum[H][8];
  __shared__ float mm[kSimtWarps][H], ll[kSimtWarps][H];
  __shared__ __align__(16) float ps[kSimtWarps][32][H];
  extern __shared__ __align__(16) uint8_t staged[];  // [warp][2 sub-blocks]; at the end the warps' outputs
  const int t = blockIdx.x, hq = blockIdx.y * H, d = a.d, n = d / 32;
  const int h = hq / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  // the request of token t: rows that no request owns, or one whose rows leave q, stay as they are
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int begin = a.cu[lo], end = a.cu[lo + 1];
  if (begin < 0 || t < begin || t >= end || end > a.T) return;
  const long long held = min((long long)max(a.lens[lo], 0), (long long)a.max_pages << a.page_shift);
  const int keys = (int)max(0LL, held - (end - 1 - t));  // keys 0 .. keys - 1 are seen
  // this CTA's keys
  const int splits = min((int)gridDim.z, max(1, (keys + 127) / 128)), z = blockIdx.z;
  if (z >= splits) return;
  const int per = ((keys + splits - 1) / splits + 31) / 32 * 32;
  const int key0 = min((long long)z * per, (long long)keys), key1 = min((long long)key0 + per, (long long)keys);
  const int* table = a.table + lo * a.table_stride;

  // The queries, and apart from them each group's sum; channel x is kept over 16^(x % 4), which code_at's factor undoes.
  // A row with an infinity has no softmax, and its scores may all be -inf, which marks hidden keys: NaN instead.
  for (int i = threadIdx.x; i < H * d; i += blockDim.x) {
    const int g = i / d, x = i - g * d;
    const float y = to_f32<T>(static_cast<const T*>(a.q)[t * a.qs[0] + (hq + g) * a.qs[1] + x]);
    q[g][x] = fabsf(y) == INFINITY ? NAN : y * a.scale;
  }
  __syncthreads();
  if (threadIdx.x < H * n) {
    const int g = threadIdx.x / n, j = threadIdx.x - g * n;
    float s = 0.f;
    for (int i = 0; i < 32; i++) s += q[g][j * 32 + i];
    qsum[g][j] = s;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < H * d; i += blockDim.x) {
    const int g = i / d, x = i - g * d;
    q[g][x] *= __uint_as_float((127u - 4u * (x & 3)) << 23);
  }
  __syncthreads();

  // Values: a lane has four channels (a half-word), lane and lane + 32 of them; a head of 32 or 64 leaves lanes over,
  // which take other keys.
  const int pieces = d / 4, at_once = pieces <= 16 ? 32 / pieces : 1;
  const int first = at_once > 1 ? lane / pieces : 0, mine = at_once > 1 ? lane % pieces : lane;
  float m[H], l[H], acc[H][2][4] = {};
#pragma unroll
  for (int g = 0; g < H; g++) m[g] = -INFINITY, l[g] = 0.f;
  // Copies a step's keys, two sub-blocks; a bit for each that lies on a page of the cache. A second step's place would
  // take the room of the CTAs that hide the copies' latency: 8 heads of 128, 100000 keys 121 us so and 127 with it,
  // 4 heads of 256, 50000 keys 74 and 99; nothing gained by more than 5%.
  const int size = staged_bytes(d), k_row = 16 * (n | 1), rest = 16 * (k_row - 16 * n), inverse = 65536 / n + 1;
  uint8_t* const own = staged + w * 2 * size;
  auto fetch = [&](int k0) {
    unsigned ok = 0;
    for (int i = 0; i < 2; i++) {
      const int key = k0 + 16 * i;
      const int page = key < key1 ? table[key >> a.page_shift] : -1;
      if (page < 0 || page >= a.n_pages) continue;
      ok |= 1u << i;
      const uint8_t* sub = a.cache +
                           c4::sub_of_slot((key & ((1 << a.page_shift) - 1)), h, a.Hkv, a.page_shift, d) +
                           (((size_t)page * a.Hkv) << (a.page_shift - 4)) * c4::sub_bytes(d);
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(own + i * size);
      for (int p = lane; p < 40 * n; p += 32) {
        const int r = (p * inverse) >> 16;  // p / n, as p < 128 where it is used
        copy16(to + (p < 16 * n ? r * k_row + (p - r * n) * 16 : 16 * p + rest), sub + 16 * p);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    return ok;
  };
  for (int k0 = key0 + w * 32; k0 < key1; k0 += kSimtWarps * 32) {
    const unsigned ok = fetch(k0);
    const int key = k0 + lane;
    float s[H];
#pragma unroll
    for (int g = 0; g < H; g++) s[g] = -INFINITY;
    if (key < key1) {
      if (ok >> (lane >> 4) & 1) {
        const uint8_t* sub = own + (lane >> 4) * size;
        const int u = lane & 15;
        const uint8_t* codes = sub + u * (k_row - 16 * n);
        sub += rest;
#pragma unroll
        for (int g = 0; g < H; g++) s[g] = 0.f;
        for (int j = 0; j < n; j++) {
          float part[H] = {};
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + c4::k_word(u, j, c, n));
#pragma unroll
            for (int half = 0; half < 2; half++) {
              const uint32_t four = word >> (16 * half);
              const float c0 = code_at(four, 0), c1 = code_at(four, 1), c2 = code_at(four, 2), c3 = code_at(four, 3);
#pragma unroll
              for (int g = 0; g < H; g++) {
                const float4 x = *reinterpret_cast<const float4*>(&q[g][32 * j + 8 * c + 4 * half]);
                part[g] = fmaf(c3, x.w, fmaf(c2, x.z, fmaf(c1, x.y, fmaf(c0, x.x, part[g]))));
              }
            }
          }
          const float sc = __half2float(*reinterpret_cast<const __half*>(sub + c4::ks_at(d) + (u * n + j) * 2));
          const float mn = __half2float(*reinterpret_cast<const __half*>(sub + c4::km_at(d) + (u * n + j) * 2));
#pragma unroll
          for (int g = 0; g < H; g++) s[g] = fmaf(part[g], sc, fmaf(qsum[g][j], mn, s[g]));
        }
      } else {
#pragma unroll
        for (int g = 0; g < H; g++) s[g] = NAN;  // a page outside the cache
      }
    }
#pragma unroll
    for (int g = 0; g < H; g++) {
      float mx = s[g];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = fmaxf(m[g], mx);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float p = expf(s[g] - base), alpha = expf(m[g] - base);
      m[g] = mx;
      l[g] = fmaf(l[g], alpha, p);
      ps[w][lane][g] = p;
#pragma unroll
      for (int e = 0; e < 2; e++)
#pragma unroll
        for (int i = 0; i < 4; i++) acc[g][e][i] *= alpha;
    }
    __syncwarp();
    const int count = min(32, key1 - k0);
#pragma unroll 4
    for (int k = first; k < count; k += at_once) {
      if (!(ok >> (k >> 4) & 1)) continue;
      const uint8_t* sk = own + (k >> 4) * size + rest;
      float pk[H];
#pragma unroll
      for (int g = 0; g < H; g++) pk[g] = ps[w][k][g];
      const int row = c4::v_row(k & 15);
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int pc = mine + 32 * e;
        if (pc < pieces) {
          const int j = pc >> 3;
          const uint32_t word = *reinterpret_cast<const uint16_t*>(sk + c4::vc_at(d) + c4::v_piece(row, j, pc & 7, n));
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(sk + c4::vp_at(d) + (row * n + j) * 4));
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float v = fmaf(code_at(word >> (4 * i), 0), sm.x, sm.y);
#pragma unroll
            for (int g = 0; g < H; g++) acc[g][e][i] = fmaf(pk[g], v, acc[g][e][i]);
          }
        }
      }
    }
    __syncwarp();  // this step's keys and weights are read
  }
  __syncthreads();
  float* const om = reinterpret_cast<float*>(staged);  // [warp][H][d]
#pragma unroll
  for (int g = 0; g < H; g++) {
    const float sum = warp_sum(l[g]);
    if (lane == 0) {
      mm[w][g] = m[g];
      ll[w][g] = sum;
    }
    for (int o = 32 / at_once; o < 32; o *= 2)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[g][0][i] += __shfl_xor_sync(0xffffffffu, acc[g][0][i], o);
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const int pc = mine + 32 * e;
      if (pc < pieces && first == 0)
#pragma unroll
        for (int i = 0; i < 4; i++) om[(w * H + g) * d + 4 * pc + i] = acc[g][e][i];
    }
  }
  __syncthreads();
  const size_t row = (size_t)t * a.Hq + hq;  // the first head's row
  const size_t parts = (size_t)a.T * a.Hq * gridDim.z;
  float* part_ml = a.part_o + parts * d;
  for (int g = 0; g < H; g++) {
    float M = -INFINITY, L = 0.f, f[kSimtWarps];
    for (int i = 0; i < kSimtWarps; i++) M = fmaxf(M, mm[i][g]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int i = 0; i < kSimtWarps; i++) {
      f[i] = expf(mm[i][g] - base);
      L = fmaf(ll[i][g], f[i], L);
    }
    // a row that sees no key has L = 0: its output is 0 and its log-sum-exp -inf
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t part = (row + g) * gridDim.z + z;
    for (int x = threadIdx.x; x < d; x += blockDim.x) {
      float o = 0.f;
      for (int i = 0; i < kSimtWarps; i++) o = fmaf(om[(i * H + g) * d + x], f[i], o);
      if (splits > 1)
        a.part_o[part * d + x] = o;
      else
        static_cast<T*>(a.o)[(row + g) * d + x] = from_f32<T>(o * inv);
    }
    if (threadIdx.x == 0) {
      if (splits > 1) {
        part_ml[2 * part] = M;
        part_ml[2 * part + 1] = L;
      } else if (a.lse) {
        a.lse[(size_t)(hq + g) * a.T + t] = L == 0.f ? -INFINITY : base + logf(L);
      }
    }
  }
  if (splits == 1) return;

  __threadfence();
  __syncthreads();
  __shared__ int joins;
  if (threadIdx.x == 0) {
    joins = (int)atomicAdd(a.counters + row / H, 1u) == splits - 1;
    if (joins) a.counters[row / H] = 0u;  // ready for the next call
  }
  __syncthreads();
  if (!joins) return;
  __threadfence();
  // a part a thread: its weight; then the sums over the parts, in order
  static_assert(kSimtSplits <= kSimtWarps * 32, "a thread a part");
  __shared__ float weight[kSimtSplits], sum[kSimtSplits];
  const int p = threadIdx.x;
  for (int g = 0; g < H; g++) {
    const float* ml = part_ml + (row + g) * gridDim.z * 2;
    __syncthreads();
    if (p < splits) weight[p] = __ldcg(ml + 2 * p);
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < splits; i++) M = fmaxf(M, weight[i]);
    const float top = M == -INFINITY ? 0.f : M;
    __syncthreads();
    if (p < splits) {
      weight[p] = expf(weight[p] - top);
      sum[p] = __ldcg(ml + 2 * p + 1);
    }
    __syncthreads();
    for (int i = 0; i < splits; i++) L = fmaf(sum[i], weight[i], L);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float* from = a.part_o + (row + g) * gridDim.z * d;
    for (int x = threadIdx.x; x < d; x += blockDim.x) {
      float o = 0.f;
#pragma unroll 8
      for (int i = 0; i < splits; i++) o = fmaf(__ldcg(from + (size_t)i * d + x), weight[i], o);
      static_cast<T*>(a.o)[(row + g) * d + x] = from_f32<T>(o * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(size_t)(hq + g) * a.T + t] = L == 0.f ? -INFINITY : top + logf(L);
  }
}

template <int H>
cudaError_t run_simt(const Cache4AttnArgs& a, bool bf16, long long most, cudaStream_t st) {
  // few rows: so many splits that about eight CTAs an SM have keys, if the table's width allows
  const long long rows = (long long)a.T * (a.Hq / H);
  long long splits = rows >= kCache4SimtCtas ? 1 : (kCache4SimtCtas + rows - 1) / rows;
  if (splits > most) splits = most;
  if (splits > kSimtSplits) splits = kSimtSplits;
  const dim3 grid(a.T, a.Hq / H, (unsigned)splits);
  auto kernel = bf16 ? cache4_attn_simt_kernel<__nv_bfloat16, H> : cache4_attn_simt_kernel<float, H>;
  const int bytes = kSimtWarps * 2 * staged_bytes(a.d);
  // set on every call: it is per device, and costs no synchronisation
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kSimtWarps * 32, bytes, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache4_attn_simt(const Cache4AttnArgs& a, bool bf16, cudaStream_t st) {
  const long long most = (((long long)a.max_pages << a.page_shift) + 127) / 128;
  // Heads share a CTA, and with it the decoding of the codes, where that leaves two CTAs with keys an SM. Alone / four
  // together, 32 heads on 8 of 128: 5000 keys 35 / 30 us, 1000 keys 13 / 20; 4 heads on one, 30000 keys 31 / 49.
  // Two together where four are too many: 4 requests of 1000 keys, 32 heads on 8: 24 alone, 19, and 25 with four.
  const int group = a.Hq / a.Hkv;
  const long long blocks = (long long)a.T * a.Hq * (most < kSimtSplits ? most : kSimtSplits);
  if (group % 4 == 0 && blocks / 4 >= 2 * 148) return run_simt<4>(a, bf16, most, st);
  if (group % 2 == 0 && blocks / 2 >= 2 * 148) return run_simt<2>(a, bf16, most, st);
  return run_simt<1>(a, bf16, most, st);
}

}  // namespace s2
