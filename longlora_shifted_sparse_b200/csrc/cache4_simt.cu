// Attention over the 4-bit cache on the CUDA cores: every type and head dim, fp32 arithmetic.
//
// o = softmax(q k^T * scale) v for one (token, query head) per CTA, over the keys up to the
// token's own place. Online softmax: each of four warps takes 32 keys at a time, a key a lane
// for the scores (a group's products with the codes are summed first, its scale and minimum
// applied once), then a few channels a lane for the values; the warps' (maximum, sum, output)
// are joined at the end. Keys the mask hides are never added, whatever their slots hold.
//
// Bound by instructions (about ten a value). Few rows are split over the keys, so that the calls
// that have them fill the GPU too: at least 128 keys a CTA, the parts joined by the last of a row's CTAs
// to arrive, in order. fp32 on a B200: 100000 keys of one head of 64: 7796 us without the split, 87 with it;
// 1000 keys, 32 heads on 32 of 128: 86 and 19; 4 requests of up to 4000, 64 on 8 of 96: 347 and 137.
#include <math.h>

#include "cache4.cuh"
#include "common.cuh"
#include "serve.h"

namespace s2 {

constexpr int kSimtWarps = 4, kSimtSplits = 128;

template <typename T>
__global__ void __launch_bounds__(kSimtWarps * 32) cache4_attn_simt_kernel(
    const __grid_constant__ Cache4AttnArgs a) {
  __shared__ float q[256], qsum[8];
  __shared__ float om[kSimtWarps][256], mm[kSimtWarps], ll[kSimtWarps];
  const int t = blockIdx.x, hq = blockIdx.y, d = a.d, n = d / 32;
  const int h = hq / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  // the request of token t: rows that no request owns stay as they are
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int begin = a.cu[lo], end = a.cu[lo + 1];
  if (t < begin || t >= end) return;
  const long long held = min((long long)max(a.lens[lo], 0), (long long)a.max_pages << a.page_shift);
  const int keys = (int)max(0LL, held - (end - 1 - t));  // keys 0 .. keys - 1 are seen
  // this CTA's keys
  const int splits = min((int)gridDim.z, max(1, (keys + 127) / 128)), z = blockIdx.z;
  if (z >= splits) return;
  const int per = ((keys + splits - 1) / splits + 31) / 32 * 32;
  const int key0 = min((long long)z * per, (long long)keys), key1 = min((long long)key0 + per, (long long)keys);
  const int* table = a.table + lo * a.table_stride;

  for (int x = threadIdx.x; x < d; x += blockDim.x)
    q[x] = to_f32<T>(static_cast<const T*>(a.q)[t * a.qs[0] + hq * a.qs[1] + x]) * a.scale;
  __syncthreads();
  if (threadIdx.x < n) {
    float s = 0.f;
    for (int i = 0; i < 32; i++) s += q[threadIdx.x * 32 + i];
    qsum[threadIdx.x] = s;
  }
  __syncthreads();

  const int pieces = d / 4;  // half-words of four channels: lane's are lane, lane + 32
  float m = -INFINITY, l = 0.f, acc[2][4] = {};
  for (int k0 = key0 + w * 32; k0 < key1; k0 += kSimtWarps * 32) {
    const int key = k0 + lane;
    float s = -INFINITY;
    const uint8_t* sub = nullptr;
    if (key < key1) {
      const int page = table[key >> a.page_shift];
      if (page >= 0 && page < a.n_pages) {
        sub = a.cache + c4::sub_of_slot((key & ((1 << a.page_shift) - 1)), h, a.Hkv, a.page_shift, d) +
              (((size_t)page * a.Hkv) << (a.page_shift - 4)) * c4::sub_bytes(d);
        const int u = key & 15;
        s = 0.f;
        for (int j = 0; j < n; j++) {
          float part = 0.f;
          for (int c = 0; c < 4; c++) {
            const uint32_t word = *reinterpret_cast<const uint32_t*>(sub + c4::k_word(u, j, c, n));
#pragma unroll
            for (int i = 0; i < 8; i++)
              part = fmaf((float)((word >> (4 * i)) & 15u), q[32 * j + 8 * c + i], part);
          }
          const float sc = __half2float(*reinterpret_cast<const __half*>(sub + c4::ks_at(d) + (u * n + j) * 2));
          const float mn = __half2float(*reinterpret_cast<const __half*>(sub + c4::km_at(d) + (u * n + j) * 2));
          s = fmaf(part, sc, fmaf(qsum[j], mn, s));
        }
      } else {
        s = NAN;  // a page outside the cache
      }
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mx = fmaxf(m, mx);
    const float base = mx == -INFINITY ? 0.f : mx;
    const float p = expf(s - base), alpha = expf(m - base);
    m = mx;
    l = fmaf(l, alpha, p);
#pragma unroll
    for (int e = 0; e < 2; e++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[e][i] *= alpha;
    const int count = min(32, key1 - k0);
    for (int k = 0; k < count; k++) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      const uint8_t* sk = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(sub), k));
      if (!sk) continue;
      const int row = c4::v_row((k0 + k) & 15);
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int pc = lane + 32 * e;
        if (pc < pieces) {
          const int j = pc >> 3, g = pc & 7;
          const uint32_t word = *reinterpret_cast<const uint16_t*>(sk + c4::vc_at(d) + c4::v_piece(row, j, g, n));
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(sk + c4::vp_at(d) + (row * n + j) * 4));
#pragma unroll
          for (int i = 0; i < 4; i++)
            acc[e][i] = fmaf(pk, fmaf((float)((word >> (4 * i)) & 15u), sm.x, sm.y), acc[e][i]);
        }
      }
    }
  }
  l = warp_sum(l);
  if (lane == 0) {
    mm[w] = m;
    ll[w] = l;
  }
#pragma unroll
  for (int e = 0; e < 2; e++) {
    const int pc = lane + 32 * e;
    if (pc < pieces)
#pragma unroll
      for (int i = 0; i < 4; i++) om[w][32 * (pc >> 3) + 4 * (pc & 7) + i] = acc[e][i];
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, f[kSimtWarps];
  for (int i = 0; i < kSimtWarps; i++) M = fmaxf(M, mm[i]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int i = 0; i < kSimtWarps; i++) {
    f[i] = expf(mm[i] - base);
    L = fmaf(ll[i], f[i], L);
  }
  if (splits > 1) {
    const size_t row = (size_t)t * a.Hq + hq, rows = (size_t)a.T * a.Hq;
    float* part = a.part_o + (row * gridDim.z + z) * d;
    float* ml = a.part_o + rows * gridDim.z * d + row * gridDim.z * 2;
    for (int x = threadIdx.x; x < d; x += blockDim.x) {
      float o = 0.f;
      for (int i = 0; i < kSimtWarps; i++) o = fmaf(om[i][x], f[i], o);
      part[x] = o;
    }
    if (threadIdx.x == 0) {
      ml[2 * z] = M;
      ml[2 * z + 1] = L;
    }
    __threadfence();
    __syncthreads();
    __shared__ int joins;
    if (threadIdx.x == 0) {
      joins = (int)atomicAdd(a.counters + row, 1u) == splits - 1;
      if (joins) a.counters[row] = 0u;  // ready for the next call
    }
    __syncthreads();
    if (!joins) return;
    __threadfence();
    // a part a thread: its weight; then the sums over the parts, in order
    static_assert(kSimtSplits <= kSimtWarps * 32, "a thread a part");
    __shared__ float weight[kSimtSplits], sum[kSimtSplits];
    const int mine = threadIdx.x;
    if (mine < splits) weight[mine] = __ldcg(ml + 2 * mine);
    __syncthreads();
    M = -INFINITY;
    for (int i = 0; i < splits; i++) M = fmaxf(M, weight[i]);
    const float top = M == -INFINITY ? 0.f : M;
    __syncthreads();
    if (mine < splits) {
      weight[mine] = expf(weight[mine] - top);
      sum[mine] = __ldcg(ml + 2 * mine + 1);
    }
    __syncthreads();
    L = 0.f;
    for (int i = 0; i < splits; i++) L = fmaf(sum[i], weight[i], L);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float* parts = a.part_o + row * gridDim.z * d;
    for (int x = threadIdx.x; x < d; x += blockDim.x) {
      float o = 0.f;
#pragma unroll 8
      for (int i = 0; i < splits; i++) o = fmaf(__ldcg(parts + (size_t)i * d + x), weight[i], o);
      static_cast<T*>(a.o)[row * d + x] = from_f32<T>(o * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(size_t)hq * a.T + t] = L == 0.f ? -INFINITY : top + logf(L);
    return;
  }
  // a row that sees no key has L = 0: its output is 0 and its log-sum-exp -inf
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int x = threadIdx.x; x < d; x += blockDim.x) {
    float o = 0.f;
    for (int i = 0; i < kSimtWarps; i++) o = fmaf(om[i][x], f[i], o);
    static_cast<T*>(a.o)[((size_t)t * a.Hq + hq) * d + x] = from_f32<T>(o * inv);
  }
  if (a.lse && threadIdx.x == 0) a.lse[(size_t)hq * a.T + t] = L == 0.f ? -INFINITY : base + logf(L);
}

cudaError_t launch_cache4_attn_simt(const Cache4AttnArgs& a, bool bf16, cudaStream_t st) {
  // few rows: so many splits that about eight CTAs an SM have keys, if the table's width allows
  const long long rows = (long long)a.T * a.Hq, most = (((long long)a.max_pages << a.page_shift) + 127) / 128;
  long long splits = rows >= kCache4SimtCtas ? 1 : (kCache4SimtCtas + rows - 1) / rows;
  if (splits > most) splits = most;
  if (splits > kSimtSplits) splits = kSimtSplits;
  const dim3 grid(a.T, a.Hq, (unsigned)splits);
  if (bf16)
    cache4_attn_simt_kernel<__nv_bfloat16><<<grid, kSimtWarps * 32, 0, st>>>(a);
  else
    cache4_attn_simt_kernel<float><<<grid, kSimtWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace s2
