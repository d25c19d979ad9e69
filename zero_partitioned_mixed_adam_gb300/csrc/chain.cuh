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

// The value that a function of the sizes has, from the last few that this thread asked for:
// what it takes to work one out is host time of every call.
template <typename Key, typename Value>
struct Memo {
  static constexpr int kKept = 8;
  Key keys[kKept];
  Value values[kKept];
  int used = 0, next = 0;
  template <typename F>
  const Value& get(const Key& key, F f) {
    for (int k = 0; k < used; ++k)
      if (keys[k] == key) return values[k];
    const int at = next;
    next = (next + 1) % kKept;
    if (used < kKept) ++used;
    keys[at] = key;
    values[at] = f();
    return values[at];
  }
};

// Lets a kernel use `bytes` of dynamic shared memory on the current device, once a thread.
inline cudaError_t allow_shared(const void* kernel, int bytes) {
  struct Allowed {
    const void* kernel;
    int device, bytes;
  };
  constexpr int kMost = 64;
  static thread_local Allowed known[kMost];
  static thread_local int count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  for (int k = 0; k < count; ++k)
    if (known[k].kernel == kernel && known[k].device == device && known[k].bytes >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && count < kMost) known[count++] = {kernel, device, bytes};
  return e;
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
