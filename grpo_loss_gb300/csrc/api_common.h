// What the translation units of the C ABI share: kernel timing around each
// launch, the NVTX range of a call, and small host helpers.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "../../include/grpo.h"

namespace grpo {

// Bracket one launch with the profiler's events (a no-op while it is off).
void prof_begin(int kind, cudaStream_t s);
void prof_end(cudaStream_t s);

// SM count of the current device (cached).
grpo_status device_info(int* sms);

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned_to(const void* p, size_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

#define LAUNCH(kind, stream, call)         \
  do {                                     \
    prof_begin(kind, stream);              \
    cudaError_t e_ = (call);               \
    prof_end(stream);                      \
    if (e_ != cudaSuccess) return GRPO_ERR_CUDA; \
  } while (0)

// NVTX range around one library call (visible in Nsight Systems timelines;
// a no-op when no tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

}  // namespace grpo
