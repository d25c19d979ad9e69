// chain.cuh -- the launches of one call as a chain of programmatic dependents, and
// the pieces of its workspace.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "linear_plan.hpp"

namespace zeroadam {
namespace {

inline bool aligned(const void* p, uintptr_t k) {
  return (reinterpret_cast<uintptr_t>(p) & (k - 1)) == 0;
}

// Takes pieces of the workspace in order.
struct Space {
  char* at;
  void* take(int64_t bytes) {
    void* p = at;
    at += round_up(bytes, 256);
    return p;
  }
};

// The kernels of one call, launched as programmatic dependents: they begin while
// their predecessor ends, and wait for it (wait_for_predecessor) before they read
// what it wrote; the first one so after whatever the stream held before.
struct Chain {
  cudaStream_t stream;
  bool begun = false;

  template <typename... Params, typename... Args>
  cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster,
                     Args&&... args) {
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    cudaLaunchAttribute attr[2];
    config.attrs = attr;
    if (cluster > 1) {
      cudaLaunchAttribute& a = attr[config.numAttrs++];
      a.id = cudaLaunchAttributeClusterDimension;
      a.val.clusterDim.x = cluster;
      a.val.clusterDim.y = 1;
      a.val.clusterDim.z = 1;
    }
    cudaLaunchAttribute& a = attr[config.numAttrs++];
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    begun = true;
    return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...);
  }
};

}  // namespace
}  // namespace zeroadam
