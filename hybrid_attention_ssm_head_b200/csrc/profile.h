// Optional per-step timing with CUDA events (hymba_profile_enable): a ProfScope around the
// launches of one pipeline step records an event on each side of them on their stream.
#pragma once

#include <cuda_runtime.h>

#include <mutex>
#include <vector>

#include "kernels.h"

namespace hymba {

struct ProfRecord {
  const char *name;
  cudaEvent_t start, stop;
  unsigned long long kernels;
};
struct Profiler {
  std::mutex mu;
  bool on = false;
  std::vector<cudaEvent_t> pool;
  size_t next = 0;
  std::vector<ProfRecord> recs;
};
Profiler &prof();
// Kernel launches counted by note_launch() so far.
unsigned long long launches_noted();

class ProfScope {
 public:
  ProfScope(cudaStream_t s, const char *name) : s_(s) {
    Profiler &p = prof();
    if (!p.on) return;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) return;
    std::lock_guard<std::mutex> g(p.mu);
    if (p.next + 2 > p.pool.size()) return;  // pool exhausted: stop recording until collected
    rec_.name = name;
    launches0_ = launches_noted();
    rec_.start = p.pool[p.next++];
    rec_.stop = p.pool[p.next++];
    cudaEventRecord(rec_.start, s_);
    active_ = true;
  }
  ~ProfScope() {
    if (!active_) return;
    cudaEventRecord(rec_.stop, s_);
    rec_.kernels = launches_noted() - launches0_;
    Profiler &p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    p.recs.push_back(rec_);
  }

 private:
  cudaStream_t s_;
  ProfRecord rec_{};
  unsigned long long launches0_ = 0;
  bool active_ = false;
};

}  // namespace hymba
