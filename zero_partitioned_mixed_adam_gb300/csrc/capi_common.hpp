// capi_common.hpp -- what the files of C entry points share: tracing, statuses,
// and the arithmetic of buffer overlaps.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

namespace zeroadam {

// Scoped NVTX range.
struct Trace {
  explicit Trace(const char* name) { nvtxRangePushA(name); }
  ~Trace() { nvtxRangePop(); }
  Trace(const Trace&) = delete;
  Trace& operator=(const Trace&) = delete;
};

// Whether zero_test_withhold_copies is on.
int withhold_copies();

// The status of a launch, keeping its CUDA error for zero_strerror.
int launch_status(cudaError_t e);

struct Range {
  uintptr_t lo, hi;
};
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline Range bytes_of(const void* p, int64_t first, int64_t count, int esize) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(first) * esize;
  return {b, b + static_cast<uintptr_t>(count) * esize};
}
inline bool nonempty(Range r) { return r.hi > r.lo; }

}  // namespace zeroadam
