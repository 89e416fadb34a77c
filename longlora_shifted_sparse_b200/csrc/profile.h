// Per-kernel event timing, shared by the files that launch kernels: the kernel ids, the
// record pool and the launch wrapper.
#pragma once

#include <cuda_runtime.h>

#include <mutex>
#include <vector>

namespace s2 {

enum KernelId {
  kRopeTable = 0,
  kRopePi,
  kFwdTc,
  kFwdSimt,
  kBwdRowsum,
  kBwdDkdvTc,
  kBwdDqTc,
  kBwdDqSimt,
  kBwdDkdvSimt,
  kRope,
  kPagePlan,
  kCache4Append,
  kCache4Read,
  kCache4Attn,
  kCache4Tc,
  kCache4AttnSimt,
  kNumKernels
};

inline const char* const kKernelNames[kNumKernels] = {
    "rope_table", "rope_pi", "fwd_tc", "fwd_simt", "bwd_rowsum", "bwd_dkdv_tc", "bwd_dq_tc",
    "bwd_dq_simt", "bwd_dkdv_simt", "rope", "page_plan", "cache4_append", "cache4_read",
    "cache4_attn", "cache4_tc", "cache4_attn_simt"};

struct Record {
  int id;
  cudaEvent_t start, stop;
};

constexpr size_t kMaxRecords = 8192;

struct Profiler {
  std::mutex mu;
  bool on = false;
  int dropped = 0;
  std::vector<Record> pending;
  std::vector<cudaEvent_t> pool;
  int launches[kNumKernels] = {};
  double total_ms[kNumKernels] = {};

  cudaEvent_t get_event() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
    return e;
  }

  // Folds finished records into the totals; returns the first CUDA error seen.
  cudaError_t drain() {
    cudaError_t first = cudaSuccess;
    for (auto& r : pending) {
      float ms = 0.f;
      cudaError_t e = cudaEventSynchronize(r.stop);
      if (e == cudaSuccess) e = cudaEventElapsedTime(&ms, r.start, r.stop);
      if (e == cudaSuccess) {
        launches[r.id] += 1;
        total_ms[r.id] += ms;
      } else if (first == cudaSuccess) {
        first = e;
      }
      pool.push_back(r.start);
      pool.push_back(r.stop);
    }
    pending.clear();
    return first;
  }
};

inline Profiler& profiler() {
  static Profiler* p = new Profiler();  // never destroyed: events may outlive static teardown
  return *p;
}

// Launches `fn` on `st`; when profiling is on, brackets it with events on the same stream.
template <typename F>
cudaError_t timed_launch(int id, cudaStream_t st, F fn) {
  Profiler& pr = profiler();
  cudaEvent_t a = nullptr, b = nullptr;
  {
    std::lock_guard<std::mutex> lk(pr.mu);
    if (pr.on) {
      if (pr.pending.size() < kMaxRecords) {
        a = pr.get_event();
        b = pr.get_event();
        if (!a || !b) {
          if (a) pr.pool.push_back(a);
          if (b) pr.pool.push_back(b);
          a = b = nullptr;
          pr.dropped++;
        }
      } else {
        pr.dropped++;
      }
    }
  }
  if (a && cudaEventRecord(a, st) != cudaSuccess) return cudaGetLastError();
  cudaError_t e = fn();
  if (e != cudaSuccess) return e;
  if (a) {
    if (cudaEventRecord(b, st) != cudaSuccess) return cudaGetLastError();
    std::lock_guard<std::mutex> lk(pr.mu);
    pr.pending.push_back(Record{id, a, b});
  }
  return cudaSuccess;
}

}  // namespace s2
