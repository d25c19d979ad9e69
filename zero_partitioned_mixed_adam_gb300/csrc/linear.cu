// linear.cu -- a unit's linear maps, forward and backward, on sm_103a.
#include "internal.h"
#include "linear_epilogue.cuh"
#include "train_ops.cuh"

namespace zeroadam {
namespace {

// D[i,j] = sum over k of A(i,k) B(j,k), each operand with a stride of its own
// along both axes: the three products of a linear map are this one.
struct Product {
  const uint16_t* a;
  int64_t a_row, a_k;
  const uint16_t* b;
  int64_t b_row, b_k;
  int64_t rows, cols, depth;
  Epilogue e;
};

constexpr int kTileM = 64, kTileN = 64, kTileK = 16;

// The plainest tiled product: 64 x 64 of D per block, 4 x 4 of it per thread,
// fp32 fused multiply-adds on values staged in shared memory.
__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ Product p) {
  __shared__ float sa[kTileK][kTileM + 4], sb[kTileK][kTileN + 4];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kTileM;
  const int64_t j0 = static_cast<int64_t>(blockIdx.y) * kTileN;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.depth; k0 += kTileK) {
    for (int q = threadIdx.x; q < kTileM * kTileK; q += 256) {
      // consecutive threads along the unit stride
      const int ka = p.a_k == 1 ? q % kTileK : q / kTileM, ia = p.a_k == 1 ? q / kTileK : q % kTileM;
      const int kb = p.b_k == 1 ? q % kTileK : q / kTileN, jb = p.b_k == 1 ? q / kTileK : q % kTileN;
      sa[ka][ia] = i0 + ia < p.rows && k0 + ka < p.depth
                       ? bf16_at(p.a + (i0 + ia) * p.a_row + (k0 + ka) * p.a_k) : 0.0f;
      sb[kb][jb] = j0 + jb < p.cols && k0 + kb < p.depth
                       ? bf16_at(p.b + (j0 + jb) * p.b_row + (k0 + kb) * p.b_k) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTileK; ++k) {
      float x[4], y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] = sa[k][ti * 4 + q];
        y[q] = sb[k][tj * 4 + q];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(x[r], y[c], acc[r][c]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t i = i0 + ti * 4 + r, j = j0 + tj * 4 + c;
      if (i < p.rows && j < p.cols) epilogue_element(p.e, i, j, acc[r][c]);
    }
}

cudaError_t launch_product(const Product& p, cudaStream_t stream) {
  const int64_t gx = (p.rows + kTileM - 1) / kTileM, gy = (p.cols + kTileN - 1) / kTileN;
  if (gx > INT32_MAX || gy > 65535) return cudaErrorInvalidValue;
  product_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// dz = bf16(dy * act'(pre)), and each column's sum of it before the rounding.
// A block takes 32 columns and all rows, 8 at a time.
struct SlopeArgs {
  const uint16_t *dy, *pre;
  int64_t ldy, ldp, rows, cols;
  int32_t act;
  uint16_t* dz;  // NULL: sums only
  int64_t ldz;
  void* dbias;   // NULL: dz only
  int32_t out_f32, accumulate;
};

__global__ void __launch_bounds__(256) slope_kernel(const __grid_constant__ SlopeArgs a) {
  __shared__ float part[8][32];
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
  const int r = threadIdx.x / 32;
  float sum = 0.0f;
  if (j < a.cols) {
    for (int64_t i = r; i < a.rows; i += 8) {
      float x = bf16_at(a.dy + i * a.ldy + j);
      if (a.act != ZERO_ACT_NONE) x *= act_slope(bf16_at(a.pre + i * a.ldp + j), a.act);
      if (a.dz != nullptr) a.dz[i * a.ldz + j] = to_bf16(x);
      sum += x;
    }
  }
  part[r][threadIdx.x % 32] = sum;
  __syncthreads();
  if (r != 0 || j >= a.cols || a.dbias == nullptr) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) sum += part[k][threadIdx.x];
  if (a.out_f32) {
    float* o = static_cast<float*>(a.dbias) + j;
    *o = a.accumulate ? *o + sum : sum;
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.dbias) + j;
    *o = to_bf16(a.accumulate ? bf16_at(o) + sum : sum);
  }
}

int64_t round_up(int64_t x, int64_t k) { return (x + k - 1) / k * k; }

}  // namespace

int64_t linear_workspace(const zero_linear_t& s, bool backward) {
  if (!backward) return 0;
  return round_up(s.rows * round_up(s.out, 8) * 2, 256);
}

cudaError_t launch_linear_forward(const LinearForwardLaunch& L) {
  (void)cudaGetLastError();
  const zero_linear_t& s = L.s;
  Product p{};
  p.a = L.x;
  p.a_row = s.ldx;
  p.a_k = 1;
  p.b = L.w;
  p.b_row = s.ldw;
  p.b_k = 1;
  p.rows = s.rows;
  p.cols = s.out;
  p.depth = s.in;
  p.e.bias = L.bias;
  p.e.act = L.act;
  p.e.pre = L.pre;
  p.e.ldp = s.ldp;
  p.e.residual = L.residual;
  p.e.ldr = s.ldr;
  p.e.out = L.y;
  p.e.ldo = s.ldy;
  return launch_product(p, L.stream);
}

cudaError_t launch_linear_backward(const LinearBackwardLaunch& L) {
  (void)cudaGetLastError();
  const zero_linear_t& s = L.s;
  const uint16_t* dz = L.dy;
  int64_t ldz = s.ldy;
  if (L.act != ZERO_ACT_NONE || L.dbias != nullptr) {
    SlopeArgs a{L.dy, L.pre, s.ldy, s.ldp, s.rows, s.out, L.act, nullptr, 0, L.dbias,
                L.grad_f32, L.accumulate};
    if (L.act != ZERO_ACT_NONE && (L.dx != nullptr || L.dw != nullptr)) {
      a.dz = static_cast<uint16_t*>(L.workspace);
      a.ldz = round_up(s.out, 8);
      dz = a.dz;
      ldz = a.ldz;
    }
    slope_kernel<<<static_cast<unsigned>((s.out + 31) / 32), 256, 0, L.stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (L.dx != nullptr && s.rows > 0) {
    Product p{};
    p.a = dz;
    p.a_row = ldz;
    p.a_k = 1;
    p.b = L.w;
    p.b_row = 1;
    p.b_k = s.ldw;
    p.rows = s.rows;
    p.cols = s.in;
    p.depth = s.out;
    p.e.slope_act = L.act_in;
    p.e.slope_of = L.act_in != ZERO_ACT_NONE ? L.pre_in : nullptr;
    p.e.lds = s.ldpi;
    p.e.out = L.dx;
    p.e.ldo = s.lddx;
    const cudaError_t e = launch_product(p, L.stream);
    if (e != cudaSuccess) return e;
  }
  if (L.dw != nullptr) {
    Product p{};
    p.a = dz;
    p.a_row = 1;
    p.a_k = ldz;
    p.b = L.x;
    p.b_row = 1;
    p.b_k = s.ldx;
    p.rows = s.out;
    p.cols = s.in;
    p.depth = s.rows;
    p.e.out = L.dw;
    p.e.ldo = s.lddw;
    p.e.out_f32 = L.grad_f32;
    p.e.accumulate = L.accumulate;
    return launch_product(p, L.stream);
  }
  return cudaSuccess;
}

}  // namespace zeroadam
