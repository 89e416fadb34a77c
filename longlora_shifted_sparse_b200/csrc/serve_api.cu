// extern "C" entry points of the serving operators: argument checks and launches.
#include <math.h>
#include <stdint.h>

#include "../../include/s2attn.h"
#include "cache4.cuh"
#include "profile.h"
#include "serve.h"

namespace s2 {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool dtype_ok(int dt) { return dt == S2_BF16 || dt == S2_FP32; }
bool headdim32_ok(int d) { return d >= 32 && d <= 256 && d % 32 == 0; }
s2_status to_status(cudaError_t e) { return e == cudaSuccess ? S2_OK : S2_ERR_CUDA; }

// log2 of a page size of 16..256 tokens, or -1.
int page_shift(int page_size) {
  for (int s = 4; s <= 8; s++)
    if (page_size == 1 << s) return s;
  return -1;
}

// Strides of rows that are read in 16-byte pieces.
bool strides16(const long long* s, int count, int dt) {
  const int v = dt == S2_BF16 ? 8 : 4;
  for (int i = 0; i < count; i++)
    if (s[i] % v != 0) return false;
  return true;
}

// Slots are 32-bit: a cache has fewer than 2^31.
bool cache_ok(int n_pages, int page_size) {
  return n_pages > 0 && (long long)n_pages * page_size <= 0x7fffffffLL;
}

// The attention's workspace: the status word, the arrival counters, the list of joins, and the
// parts of whichever kernel runs.
constexpr size_t round256(size_t x) { return (x + 255) / 256 * 256; }
constexpr size_t kAtCounters = 256;
constexpr size_t kAtJoins =
    kAtCounters + round256((kCache4MaxCtas > kCache4SimtCtas ? kCache4MaxCtas : kCache4SimtCtas) * sizeof(unsigned));
constexpr size_t kAtParts = kAtJoins + round256(kCache4TcCtas * 2 * sizeof(int4));
constexpr size_t kPartsO = (size_t)2 * kCache4MaxCtas * kCache4PartFloats;
constexpr size_t kTcPartsO = (size_t)2 * kCache4TcCtas * kCache4TcRows * 128;
constexpr size_t kPartsFloats = kPartsO + (size_t)2 * kCache4MaxCtas * 2 * kCache4PartRows;
constexpr size_t kTcPartsFloats = kTcPartsO + (size_t)2 * kCache4TcCtas * 2 * kCache4TcRows;
constexpr size_t kCache4WsBytes =
    kAtParts + sizeof(float) * (kPartsFloats > kTcPartsFloats ? kPartsFloats : kTcPartsFloats);
static_assert((size_t)2 * kCache4SimtCtas * 4 * (256 + 2) <= kTcPartsFloats, "the splits' parts fit");

// Tensor instructions: bf16 and a head dim that is a whole number of their wide loads.
bool cache4_mma(int d, int dt) { return dt == S2_BF16 && (d == 64 || d == 128 || d == 256); }
// Tiles of 256 query rows on tcgen05, or of 8 to 32 on mma.sync? The first dequantise a key once for
// many rows; the second start sooner. `rows`: of a request and kv head; `pairs`: rows times keys of
// the whole call, at most what the block table's width allows. us, mma.sync / tcgen05, d = 128, in a table as wide as the keys:
//   1 request, 64 heads on 8, 256 keys:    64 rows 13 / 24, 512 rows 14 / 34
//   1 request, 64 heads on 8, 1024 keys:   64 rows 20 / 24, 128 rows 19 / 26, 512 rows 31 / 33
//   1 request, 64 heads on 8, 4096 keys:   32 rows 26 / 26,  64 rows 34 / 27, 512 rows 70 / 36
//   8 requests, 32 heads on 32, 4096 keys: 32 rows 127 / 143, 64 rows 225 / 147, 512 rows 1524 / 350
//   1 request, 64 heads on 8, 16384 keys:  64 rows 57 / 45, 512 rows 206 / 72
// In a table for 102400 tokens the same calls take 15 / 24, 18 / 35; 19 / 24, 24 / 26, 30 / 33; 35 / 25, 35 / 27, 70 / 36; 127 / 143, 224 / 147,
// 1524 / 351; 57 / 45, 207 / 72, and the rule, which knows the width and not the lengths, takes tcgen05 from 64 rows on: short chunks in
// wide tables pay for it, at most 35 us where 14 would do.
bool cache4_many(int d, long long rows, double pairs) {
  return (d == 64 || d == 128) && rows >= 64 && pairs >= 3.0 * (1 << 20);
}

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" {

s2_status s2attn_rope_freqs(double* turns, int rotary_dim, double rope_base, double pi_scale,
                            int original_len, double slow_turns, double fast_turns) {
  if (!turns) return S2_ERR_NULL;
  if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2) return S2_ERR_HEADDIM;
  if (!(isfinite(pi_scale) && pi_scale > 0) || !(isfinite(rope_base) && rope_base > 0) ||
      original_len < 0)
    return S2_ERR_ARG;
  if (original_len > 0 &&
      !(isfinite(slow_turns) && isfinite(fast_turns) && slow_turns >= 0 && fast_turns > slow_turns))
    return S2_ERR_ARG;
  const double two_pi = 6.283185307179586476925287;
  for (int i = 0; i < rotary_dim / 2; i++) {
    const double plain = pow(rope_base, -2.0 * i / rotary_dim) / two_pi;
    double f = plain / pi_scale;
    if (original_len > 0) {
      const double x = (plain * original_len - slow_turns) / (fast_turns - slow_turns);
      const double keep = x < 0 ? 0 : x > 1 ? 1 : x;
      f = keep * plain + (1 - keep) * f;
    }
    turns[i] = f;
  }
  return S2_OK;
}

s2_status s2attn_rope(const void* q, void* q_out, const void* k, void* k_out,
                      const void* positions, int positions64, const double* freqs, int B, int N,
                      int H_q, int H_kv, int d, int rotary_dim, const long long* q_strides,
                      const long long* k_strides, const long long* pos_strides, int layout,
                      int inverse, float mscale, int dtype, void* cuda_stream) {
  if (!q || !q_out || (!k != !k_out) || !positions || !freqs || !q_strides ||
      (k && !k_strides) || !pos_strides)
    return S2_ERR_NULL;
  if (!dtype_ok(dtype)) return S2_ERR_DTYPE;
  if (B <= 0 || N <= 0 || H_q <= 0 || (k && H_kv <= 0) || (long long)B * N > 0x7fffffffLL ||
      H_q > 65535 || (k && H_kv > 65535))
    return S2_ERR_SHAPE;
  if (d < 2 || d > 256 || d % 2 || rotary_dim < 2 || rotary_dim > d || rotary_dim % 2)
    return S2_ERR_HEADDIM;
  if ((layout != S2_ROPE_INTERLEAVED && layout != S2_ROPE_HALF) || !isfinite(mscale))
    return S2_ERR_ARG;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out))
    return S2_ERR_ALIGN;
  if (((uintptr_t)freqs & 7u) || ((uintptr_t)positions & (positions64 ? 7u : 3u)))
    return S2_ERR_ALIGN;
  RopeArgs a{};
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.pos = positions; a.pos64 = positions64 != 0; a.turns = freqs;
  a.B = B; a.N = N; a.Hq = H_q; a.Hkv = k ? H_kv : 0; a.d = d; a.rot = rotary_dim;
  a.half = layout == S2_ROPE_HALF; a.inverse = inverse != 0; a.mscale = mscale;
  const long long qd[3] = {(long long)N * H_q * d, (long long)H_q * d, d};
  const long long kd[3] = {(long long)N * H_kv * d, (long long)H_kv * d, d};
  for (int i = 0; i < 3; i++) {
    a.qs[i] = q_strides[i];
    a.qos[i] = q_out == q ? q_strides[i] : qd[i];
    if (k) {
      a.ks[i] = k_strides[i];
      a.kos[i] = k_out == k ? k_strides[i] : kd[i];
    }
  }
  a.ps[0] = pos_strides[0];
  a.ps[1] = pos_strides[1];
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return to_status(timed_launch(kRope, s, [&] { return launch_rope(a, dtype == S2_BF16, s); }));
}

s2_status s2attn_page_plan(const int* cached_lens, const int* new_lens, const int* free_pages,
                           const int* free_count, int* block_table, int* cu_new, int* lens,
                           int* positions, int* slots, int* counts, int R, int T, int n_free,
                           int max_pages, long long table_stride, int page_size,
                           void* cuda_stream) {
  if (!cached_lens || !new_lens || (!free_pages && n_free > 0) || !free_count || !block_table ||
      !cu_new || !lens || (T > 0 && (!positions || !slots)) || !counts)
    return S2_ERR_NULL;
  if (R <= 0 || R > kPlanMaxRequests || T < 0 || n_free < 0 || max_pages <= 0 ||
      table_stride < max_pages)
    return S2_ERR_SHAPE;
  const int shift = page_shift(page_size);
  if (shift < 0) return S2_ERR_ARG;
  if ((long long)max_pages << shift > 0x7fffffffLL) return S2_ERR_SHAPE;
  PlanArgs a{};
  a.cached = cached_lens; a.fresh = new_lens; a.free_pages = free_pages; a.free_count = free_count;
  a.table = block_table; a.cu_new = cu_new; a.lens = lens; a.positions = positions;
  a.slots = slots; a.counts = counts; a.table_stride = table_stride;
  a.R = R; a.T = T; a.n_free = n_free; a.max_pages = max_pages; a.page_shift = shift;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return to_status(timed_launch(kPagePlan, s, [&] { return launch_page_plan(a, s); }));
}

size_t s2attn_cache4_bytes(int n_pages, int page_size, int H_kv, int d) {
  const int shift = page_shift(page_size);
  if (shift < 0 || H_kv <= 0 || H_kv > 65535 || !headdim32_ok(d) || !cache_ok(n_pages, page_size)) return 0;
  return ((size_t)n_pages * H_kv << (shift - 4)) * c4::sub_bytes(d);
}

s2_status s2attn_cache4_append(const void* k, const void* v, void* cache, const int* slots, int T,
                               int H_kv, int d, int n_pages, int page_size,
                               const long long* k_strides, const long long* v_strides, int dtype,
                               void* cuda_stream) {
  if (!k || !v || !cache || !slots || !k_strides || !v_strides) return S2_ERR_NULL;
  if (!dtype_ok(dtype)) return S2_ERR_DTYPE;
  if (T <= 0 || H_kv <= 0 || H_kv > 65535 || (long long)T * H_kv > 0x7fffffffLL ||
      !cache_ok(n_pages, page_size))
    return S2_ERR_SHAPE;
  if (!headdim32_ok(d)) return S2_ERR_HEADDIM;
  const int shift = page_shift(page_size);
  if (shift < 0) return S2_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || !strides16(k_strides, 2, dtype) ||
      !strides16(v_strides, 2, dtype))
    return S2_ERR_ALIGN;
  RowsArgs a{};
  a.k = k; a.v = v; a.cache = static_cast<uint8_t*>(cache); a.slots = slots;
  for (int i = 0; i < 2; i++) {
    a.ks[i] = k_strides[i];
    a.vs[i] = v_strides[i];
  }
  a.n_slots = (long long)n_pages * page_size;
  a.T = T; a.Hkv = H_kv; a.d = d; a.page_shift = shift;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return to_status(
      timed_launch(kCache4Append, s, [&] { return launch_cache4_append(a, dtype == S2_BF16, s); }));
}

s2_status s2attn_cache4_read(const void* cache, const int* slots, void* k, void* v, int T,
                             int H_kv, int d, int n_pages, int page_size, int dtype,
                             void* cuda_stream) {
  if (!k || !v || !cache || !slots) return S2_ERR_NULL;
  if (!dtype_ok(dtype)) return S2_ERR_DTYPE;
  if (T <= 0 || H_kv <= 0 || H_kv > 65535 || (long long)T * H_kv > 0x7fffffffLL ||
      !cache_ok(n_pages, page_size))
    return S2_ERR_SHAPE;
  if (!headdim32_ok(d)) return S2_ERR_HEADDIM;
  const int shift = page_shift(page_size);
  if (shift < 0) return S2_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return S2_ERR_ALIGN;
  RowsArgs a{};
  a.ko = k; a.vo = v;
  a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  a.slots = slots;
  a.n_slots = (long long)n_pages * page_size;
  a.T = T; a.Hkv = H_kv; a.d = d; a.page_shift = shift;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  return to_status(
      timed_launch(kCache4Read, s, [&] { return launch_cache4_read(a, dtype == S2_BF16, s); }));
}

size_t s2attn_cache4_workspace_bytes(void) {
  return kCache4WsBytes;
}

s2_status s2attn_cache4_attn(const void* q, const void* cache, const int* block_table,
                             const int* lens, const int* cu_new, void* o, float* lse, int R, int T,
                             int H_q, int H_kv, int d, int n_pages, int page_size, int max_pages,
                             long long table_stride, const long long* q_strides, int max_new,
                             float scale, int dtype, void* workspace, size_t ws_bytes,
                             void* cuda_stream) {
  if (!q || !cache || !block_table || !lens || !cu_new || !o || !q_strides) return S2_ERR_NULL;
  if (!dtype_ok(dtype)) return S2_ERR_DTYPE;
  if (R <= 0 || T <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || H_q > 65535 || max_pages <= 0 ||
      (table_stride != 0 && table_stride < max_pages) || max_new <= 0 || (long long)T * H_q > 0x7fffffffLL ||
      !cache_ok(n_pages, page_size))
    return S2_ERR_SHAPE;
  if (!headdim32_ok(d)) return S2_ERR_HEADDIM;
  const int shift = page_shift(page_size);
  if (shift < 0 || !isfinite(scale)) return S2_ERR_ARG;
  if ((long long)max_pages << shift > 0x7fffff00LL) return S2_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(o) || !strides16(q_strides, 2, dtype))
    return S2_ERR_ALIGN;
  if (!workspace || ws_bytes < s2attn_cache4_workspace_bytes()) return S2_ERR_WORKSPACE;
  if (!aligned16(workspace)) return S2_ERR_ALIGN;
  Cache4AttnArgs a{};
  a.q = q; a.o = o; a.lse = lse; a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table; a.lens = lens; a.cu = cu_new;
  a.qs[0] = q_strides[0]; a.qs[1] = q_strides[1]; a.table_stride = table_stride;
  a.R = R; a.T = T; a.Hq = H_q; a.Hkv = H_kv; a.d = d; a.page_shift = shift;
  a.n_pages = n_pages; a.max_pages = max_pages; a.max_new = max_new; a.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool bf16 = dtype == S2_BF16;
  char* ws = static_cast<char*>(workspace);
  a.status = reinterpret_cast<unsigned*>(ws);
  a.counters = reinterpret_cast<unsigned*>(ws + kAtCounters);
  a.joins = reinterpret_cast<int4*>(ws + kAtJoins);
  a.part_o = reinterpret_cast<float*>(ws + kAtParts);
  if (cache4_mma(d, dtype)) {
    const long long rows = (long long)max_new * (H_q / H_kv);
    if (cache4_many(d, rows, (double)R * H_kv * rows * ((long long)max_pages << shift))) {
      a.part_ml = a.part_o + kTcPartsO;
      return to_status(timed_launch(kCache4Tc, s, [&] { return launch_cache4_tc(a, s); }));
    }
    a.part_ml = a.part_o + kPartsO;
    return to_status(timed_launch(kCache4Attn, s, [&] { return launch_cache4_attn(a, s); }));
  }
  return to_status(timed_launch(kCache4AttnSimt, s, [&] { return launch_cache4_attn_simt(a, bf16, s); }));
}

}  // extern "C"
