// Block tables and slot maps of one step, from the requests' lengths alone.
//
// Request r has cached[r] tokens in its pages and adds fresh[r]. Its new tokens take rows
// cu_new[r] .. of the step's token buffer, positions cached[r] .., and the slots of its pages;
// it needs ceil((cached + fresh) / P) - ceil(cached / P) pages more, taken from the end of
// the list of free pages in the requests' order. Two prefix sums (tokens, pages), then
// independent writes: every CTA forms the sums of all requests for itself in shared memory
// (at most 4096 requests, 8 bytes each, from L2) and writes its share of the outputs, so that
// one launch without a grid-wide wait does it all. Bound by latency: a few dependent loads.
//
// A request is left out (its slots are -1, its length and pages stay) where its lengths are
// negative, the table is too narrow, the token buffer ends before its tokens or the free
// pages run out. The sums are monotone, so for the last two every later request with tokens
// or pages to place is left out too, and the pages taken are one run of the list.
#include "common.cuh"
#include "serve.h"

namespace s2 {

constexpr int kPlanThreads = 256;

// Exclusive prefix sum over the block's threads, and the total.
__device__ inline long long block_prefix(long long x, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; i++) {
    if (i < w) before += warp_sums[i];
    total += warp_sums[i];
  }
  __syncthreads();
  return before + s - x;
}

// Largest r with a[r] <= x (a[0] = 0 <= x, a not decreasing, a[n] > x).
__device__ inline int find_request(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct PlanSizes {
  int tokens, pages;
  bool fits;
};

__device__ inline PlanSizes plan_sizes(const PlanArgs& a, int r, int& cached) {
  cached = a.cached[r];
  const int fresh = a.fresh[r];
  PlanSizes s{0, 0, false};
  if (cached < 0 || fresh < 0) return s;
  s.tokens = fresh;
  const long long P1 = (1 << a.page_shift) - 1;
  const long long before = (cached + P1) >> a.page_shift;
  const long long after = ((long long)cached + fresh + P1) >> a.page_shift;
  s.fits = after <= a.max_pages;
  s.pages = s.fits ? (int)(after - before) : 0;
  return s;
}

template <int E>
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int sh[];
  __shared__ long long warp_sums[kPlanThreads / 32];
  __shared__ int taken_max, left_out;
  int* tok = sh;              // [R + 1] first token row of each request
  int* page = sh + a.R + 1;   // [R] first taken page of each request
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = threadIdx.x * per, r1 = min(r0 + per, a.R);
  if (threadIdx.x == 0) taken_max = left_out = 0;
  long long nt = 0, np = 0;
  int cached;
  for (int r = r0; r < r1; r++) {
    const PlanSizes s = plan_sizes(a, r, cached);
    nt += s.tokens;
    np += s.pages;
  }
  long long total, pages;
  long long t0 = block_prefix(nt, warp_sums, total), p0 = block_prefix(np, warp_sums, pages);
  const long long kMax = 0x7fffffff;  // sums beyond it belong to requests that are left out
  const int T = (int)min(total, kMax);
  const int free_count = max(0, min(*a.free_count, a.n_free));
  const bool first = blockIdx.x == 0;
  int out = 0, took = 0;
  for (int r = r0; r < r1; r++) {
    const PlanSizes s = plan_sizes(a, r, cached);
    tok[r] = (int)min(t0, kMax);
    t0 += s.tokens;
    const bool ok = s.fits && (s.pages == 0 || p0 + s.pages <= free_count) &&
                    (s.tokens == 0 || t0 <= a.T);
    // a request that is left out keeps its tokens' rows but owns no page: bit 31 marks it
    page[r] = (int)min(p0, kMax) | (ok ? 0 : 0x80000000);
    p0 += s.pages;
    if (ok && s.pages) took = (int)p0;
    out += !ok;
    if (first) {
      a.cu_new[r] = tok[r];
      a.lens[r] = ok ? cached + s.tokens : a.cached[r];
    }
  }
  if (took) atomicMax(&taken_max, took);
  if (out) atomicAdd(&left_out, out);
  if (threadIdx.x == 0) {
    tok[a.R] = T;
  }
  __syncthreads();
  if (first && threadIdx.x == 0) {
    a.cu_new[a.R] = T;
    a.counts[0] = free_count - taken_max;
    a.counts[1] = left_out;
  }
  // E tokens a thread: one search, and one page number as long as they share a page
  const int stride = gridDim.x * kPlanThreads;
  const bool wide = (((uintptr_t)a.positions | (uintptr_t)a.slots) & 15) == 0;
  for (long long t0 = (long long)E * (blockIdx.x * kPlanThreads + threadIdx.x); t0 < a.T; t0 += (long long)E * stride) {
    int r = t0 < T ? find_request(tok, a.R, (int)t0) : 0, last = -1, base = 0;
    int pos[E], slot[E];
#pragma unroll
    for (int e = 0; e < E; e++) {
      const int t = (int)t0 + e;
      pos[e] = 0;
      slot[e] = -1;
      if (t0 + e >= min(T, a.T)) continue;
      while (t >= tok[r + 1]) {
        r++;
        last = -1;
      }
      const int c = a.cached[r];
      pos[e] = (int)((unsigned)c + (unsigned)(t - tok[r]));
      if (page[r] < 0) continue;
      const int col = pos[e] >> a.page_shift;
      if (col != last) {
        const int held = (c + (1 << a.page_shift) - 1) >> a.page_shift;
        const int p = col < held ? a.table[r * a.table_stride + col]
                                 : a.free_pages[free_count - 1 - (page[r] + col - held)];
        // a page whose slots have no 31-bit number is none: -1, not another page's slots
        base = (unsigned)p <= 0x7fffffffu >> a.page_shift ? p << a.page_shift : -1;
        last = col;
      }
      if (base >= 0) slot[e] = base + (pos[e] & ((1 << a.page_shift) - 1));
    }
    if (E == 4 && wide && t0 + 4 <= a.T) {
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[E > 1], pos[E > 2 ? 2 : 0], pos[E - 1]);
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[E > 1], slot[E > 2 ? 2 : 0], slot[E - 1]);
    } else {
#pragma unroll
      for (int e = 0; e < E; e++)
        if (t0 + e < a.T) {
          a.positions[t0 + e] = pos[e];
          a.slots[t0 + e] = slot[e];
        }
    }
  }
  // the pages' places in the table: a lane's run of the pages taken
  const int take = taken_max;
  for (int i = blockIdx.x * kPlanThreads + threadIdx.x; i < take; i += stride) {
    int lo = 0, hi = a.R;  // last request whose first page is <= i: it owns page i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((page[mid] & 0x7fffffff) <= i)
        lo = mid;
      else
        hi = mid;
    }
    const int held = (a.cached[lo] + (1 << a.page_shift) - 1) >> a.page_shift;
    a.table[lo * a.table_stride + held + (i - page[lo])] = a.free_pages[free_count - 1 - i];
  }
}

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st) {
  const size_t smem = (2 * a.R + 1) * sizeof(int);
  // Few tokens: one a thread, for latency (64 requests of a token each: 5.4 us against 8.2 with four).
  // Many: four (509 prompts, 1 M tokens: 12.3 us; one a thread on a CTA per SM took 32).
  const bool few = a.T <= 148 * kPlanThreads;
  const long long per = few ? kPlanThreads : 4 * kPlanThreads, need = (a.T + per - 1) / per;
  const int blocks = (int)(need < 1 ? 1 : need > 148 * 8 ? 148 * 8 : need);
  if (few)
    page_plan_kernel<1><<<blocks, kPlanThreads, smem, st>>>(a);
  else
    page_plan_kernel<4><<<blocks, kPlanThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace s2
