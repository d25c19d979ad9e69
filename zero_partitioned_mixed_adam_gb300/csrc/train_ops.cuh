// train_ops.cuh -- declarations shared by the C-ABI layer and the kernel files
// of the training-step operators around the optimizer step: linear maps, the
// gradient norm, AdamW over a list of tensors.  Not installed.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "zeroadam.h"

namespace zeroadam {

// ------------------------------------------------------------ tensor lists

struct NormLaunch {
  int32_t ntensors;
  const void* const* grads;
  const int64_t* numels;
  int32_t grad_f32;
  float max_norm;
  float* out;
  void* workspace;
  cudaStream_t stream;
};

// The step's scalars, each formed in double and rounded to binary32 once.
struct AdamwScalars {
  float b1, omb1, b2, omb2;  // beta1, 1 - beta1, beta2, 1 - beta2
  float size;                // lr / (1 - beta1^t)
  float inv_root;            // 1 / sqrt(1 - beta2^t)
  float eps;
};

struct AdamwLaunch {
  int32_t ntensors;
  const zero_adamw_tensor_t* tensors;
  int32_t grad_f32, eight;
  double lr;
  AdamwScalars s;
  const float* grad_scale;
  uint32_t seed;
  cudaStream_t stream;
};

struct MomentsLaunch {
  int32_t ntensors;
  const zero_adamw_tensor_t* tensors;
  float* const* m_out;  // NULL: not wanted
  float* const* v_out;
  cudaStream_t stream;
};

// Bytes of the norm's workspace: the blocks' ticket and one fp64 per block.
constexpr int64_t kNormSlots = 4096;
constexpr int64_t kNormWorkspace = 16 + 8 * kNormSlots;

cudaError_t launch_grad_norm(const NormLaunch& L);
cudaError_t launch_adamw(const AdamwLaunch& L);
cudaError_t launch_adamw_moments(const MomentsLaunch& L);

// -------------------------------------------------------------- linear maps

struct LinearForwardLaunch {
  zero_linear_t s;
  const uint16_t *x, *w, *bias, *residual;
  int32_t act;
  uint16_t *pre, *y;
  void* workspace;
  cudaStream_t stream;
  int32_t withhold;  // test hook of the bounded waits (zero_test_withhold_copies)
};

struct LinearBackwardLaunch {
  zero_linear_t s;
  const uint16_t *dy, *x, *w, *pre, *pre_in;
  int32_t act, act_in;
  uint16_t* dx;
  void *dw, *dbias;
  int32_t grad_f32, accumulate;
  void* workspace;
  cudaStream_t stream;
  int32_t withhold;
};

// flags: ZERO_LINEAR_*
int64_t linear_workspace(const zero_linear_t& s, int32_t flags);
cudaError_t launch_linear_forward(const LinearForwardLaunch& L);
cudaError_t launch_linear_backward(const LinearBackwardLaunch& L);
// Status word of the products' bounded waits on the current device (0 = every
// wait completed); read and cleared.  Returns -1 if CUDA fails.
int read_and_clear_linear_status(int* status);

}  // namespace zeroadam
