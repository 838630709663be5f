// What the linear attention kernels share: the decay's range and a sequence's length.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace hymba {

// exp(-110) is below fp32's smallest subnormal: a log decay below it, -infinity included,
// forgets the state.  Bounding it there keeps sums of log decays finite, so that their
// differences stay defined.  A NaN stays a NaN.
constexpr float kMinLogDecay = -110.f;
__device__ __forceinline__ float linear_log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }
__device__ __forceinline__ float linear_decay(float g) { return expf(linear_log_decay(g)); }

// Rows of sequence b that count.
__device__ __forceinline__ int linear_length(const hymba_linear_attention &a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.n_rows) : a.n_rows;
}

}  // namespace hymba
