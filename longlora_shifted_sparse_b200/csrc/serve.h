// Argument blocks and host-side launchers of the serving operators: rotary positions, page
// plans, and the 4-bit cache with the attention that reads it (internal; not the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace s2 {

struct RopeArgs {
  const void* q;
  const void* k;      // may be null: q alone is rotated
  void* qo;
  void* ko;
  const void* pos;    // int32 or int64
  const double* turns;  // turns per token of each pair, [rot / 2]
  int pos64, B, N, Hq, Hkv, d, rot, half, inverse;
  float mscale;
  // element strides of the inputs: batch, token, head; an output in place has its input's,
  // any other is dense
  long long qs[3], ks[3], qos[3], kos[3];
  long long ps[2];    // of the positions: batch, token
};
cudaError_t launch_rope(const RopeArgs& a, bool bf16, cudaStream_t st);

struct PlanArgs {
  const int* cached;
  const int* fresh;
  const int* free_pages;
  const int* free_count;
  int* table;
  int* cu_new;
  int* lens;
  int* positions;
  int* slots;
  int* counts;        // {free pages left, requests left out}
  long long table_stride;
  int R, T, n_free, max_pages, page_shift;
};
constexpr int kPlanMaxRequests = 4096;
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st);

struct RowsArgs {
  const void* k;      // append: inputs with strides
  const void* v;
  void* ko;           // read: dense outputs [T][Hkv][d]
  void* vo;
  uint8_t* cache;
  const int* slots;
  long long ks[2], vs[2];
  long long n_slots;  // slots of the cache: n_pages * page_size
  int T, Hkv, d, page_shift;
};
cudaError_t launch_cache4_append(const RowsArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_cache4_read(const RowsArgs& a, bool bf16, cudaStream_t st);

struct Cache4AttnArgs {
  const void* q;
  void* o;            // dense [T][Hq][d]
  float* lse;         // [Hq][T], or null
  const uint8_t* cache;
  const int* table;
  const int* lens;
  const int* cu;
  long long qs[2], table_stride;
  int R, T, Hq, Hkv, d, page_shift, n_pages, max_pages, max_new;
  float scale;
  // workspace: the status word (a bounded wait expired), arrival counters (zero between calls), the
  // list of tiles to join, and two parts a CTA: output sums, then maxima and sums of the rows
  unsigned* status;
  unsigned* counters;
  int4* joins;
  float* part_o;
  float* part_ml;
  int min_chunk;      // steps that a CTA takes at least
  int roomy;          // the grid has a CTA for every min_chunk steps that the table's width allows
};
// few rows: bf16, d = 64, 128 or 256
constexpr int kCache4MaxCtas = 148 * 4, kCache4PartRows = 32, kCache4PartFloats = 4096;
cudaError_t launch_cache4_attn(Cache4AttnArgs a, cudaStream_t st);
// many rows: bf16, d = 64 or 128
constexpr int kCache4TcCtas = 148, kCache4TcRows = 256;
cudaError_t launch_cache4_tc(Cache4AttnArgs a, cudaStream_t st);
// any type and head dim; splits of up to 2 kCache4SimtCtas parts of four heads of d + 2 floats in part_o
constexpr int kCache4SimtCtas = 148 * 8;
cudaError_t launch_cache4_attn_simt(const Cache4AttnArgs& a, bool bf16, cudaStream_t st);

}  // namespace s2
