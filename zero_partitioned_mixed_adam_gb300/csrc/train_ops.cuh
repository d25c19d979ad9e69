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
  const float* scale;  // of dx and dw, one number on the device; NULL: 1
  const float* row_scale;  // of dx, a number a row (0: dx is 0, whatever is in w); NULL: 1
  // How many of the rows there are, on the device; NULL: all.  What lies behind them in dx is
  // left anyhow; in dy and x rows up to the next multiple of 128, and least_rows, are 0.
  const int32_t* rows_now;
  uint16_t* dx_all;    // dx in its place if all rows are there; NULL: it goes to dx anyhow
  int64_t ld_all;
};
int64_t least_rows(const zero_linear_t& s, bool dx);
// Whether dx_all may be given, for a dx_all that TMA can write.
bool whole_in_place(const zero_linear_t& s, bool dw);

// ------------------------------------------- exponentials of a linear map's rows

// What becomes of z = x W^T in place of an epilogue: over each part of the columns, the
// target's left out, the sum of exp(d) and the largest z.
//   with ref      d = z - ref of its row; exp(d) is written too, in bf16, 0 for the target
//   with targets  d = z less the largest z
struct ExponentOf {
  float2* sums;           // [rows][sum_pitch], exponent_parts of them written
  int64_t sum_pitch;
  const float* ref;       // [rows]
  const int32_t* target;  // [rows], -1: none
  const int32_t* only_if; // nothing is done where this is 0; NULL: always
  const void* targets;    // [rows], as the caller gives them
  int32_t ids_i32;
  int64_t ignore;
  int32_t* ticket;        // set to 0
};
struct ExponentLaunch {
  int64_t rows, width, vocab;
  const uint16_t *x, *w;  // where TMA can read them
  int64_t ldx, ldw;
  ExponentOf of;
  uint16_t* out;          // [rows][ldo]
  int64_t ldo;
  const int32_t* rows_now;  // how many of the rows there are, on the device; NULL: all
  cudaStream_t stream;
  int32_t withhold;
};
int64_t exponent_parts(int64_t rows, int64_t vocab, int64_t width);
cudaError_t launch_exponents(const ExponentLaunch& L);

// Whether TMA can read a matrix in place; else the pitch of a copy that it can read,
// and the copy.
bool tileable_matrix(const uint16_t* p, int64_t rows, int64_t cols, int64_t ld);
int64_t laid_out_pitch(int64_t cols);
cudaError_t launch_lay_out(const uint16_t* p, int64_t rows, int64_t cols, int64_t ld, uint16_t* to,
                           cudaStream_t stream);

// ------------------------------------------------------------------ cross entropy

struct CrossEntropyLaunch {
  zero_cross_entropy_t s;
  const uint16_t *x, *w;
  const void* targets;
  int32_t ids_i32;
  int64_t ignore;
  const float* scale;
  float *losses, *total;
  uint16_t* dx;
  void* dw;
  int32_t grad_f32, accumulate;
  void* workspace;
  cudaStream_t stream;
  int32_t withhold;
};
// flags: ZERO_LINEAR_BACKWARD, ZERO_LINEAR_ALIGNED, ZERO_GRAD_F32
int64_t cross_entropy_workspace(const zero_cross_entropy_t& s, int32_t flags);
cudaError_t launch_cross_entropy(const CrossEntropyLaunch& L);

// ---------------------------------------------------------------------- embedding

struct EmbeddingLaunch {
  zero_embedding_t s;
  const uint16_t* from;   // the table, or dy
  const void* ids;
  int32_t ids_i32;
  float scale;
  int64_t padding;        // backward
  void* to;               // y, or dtable
  int32_t grad_f32, accumulate;
  cudaStream_t stream;
};
cudaError_t launch_embedding_forward(const EmbeddingLaunch& L);
cudaError_t launch_embedding_backward(const EmbeddingLaunch& L);

// -------------------------------------------------------------------- block norms

struct BlockNormLaunch {
  zero_block_norm_t s;
  const uint16_t *r, *h, *post_weight, *post_bias, *gate, *weight, *bias;
  const uint16_t *dy, *ds, *sum;   // backward: `sum` is s
  uint16_t *s_out, *y;             // forward
  uint16_t *dr, *dh;               // backward
  void *dgate, *dpost_weight, *dpost_bias, *dweight, *dbias;
  int32_t grad_f32, accumulate;
  void* workspace;
  cudaStream_t stream;
};
cudaError_t launch_block_norm_forward(const BlockNormLaunch& L);
cudaError_t launch_block_norm_backward(const BlockNormLaunch& L);
int64_t block_norm_workspace(const zero_block_norm_t& s);

// flags: ZERO_LINEAR_*
int64_t linear_workspace(const zero_linear_t& s, int32_t flags);
cudaError_t launch_linear_forward(const LinearForwardLaunch& L);
cudaError_t launch_linear_backward(const LinearBackwardLaunch& L);
// Status word of the products' bounded waits on the current device (0 = every
// wait completed); read and cleared.  Returns -1 if CUDA fails.
int read_and_clear_linear_status(int* status);

}  // namespace zeroadam
