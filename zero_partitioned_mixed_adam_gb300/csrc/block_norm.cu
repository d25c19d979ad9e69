// block_norm.cu -- the norms before and after a model's block with its gate and
// residual scale, forward and backward, on sm_103a:
//   s = r + alpha * gate * P(h),   y = N(s),
// a row at a time, in registers between its loads and its stores, so that each matrix is
// read or written once.  Bound by HBM: 8 bytes an element forward, 12 backward.
#include "chain.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

constexpr int kMostThreads = 512;

struct NormArgs {
  int64_t rows, width;
  int32_t post, kind;
  float alpha, eps;
  const uint16_t *r, *h, *w1, *b1, *gate, *w, *b;
  uint16_t *s_out, *y;
  const uint16_t *dy, *ds, *s;
  uint16_t *dr, *dh, *dgate_rows;  // dgate_rows: a matrix
  int64_t ldr, ldh, ldg, lds, ldy, lddy, ldds, lddr, lddh, lddg;
  int32_t wvec;    // the vectors are read 16 bytes at a time
  // backward: sums of each block's rows, [kSums][blocks][width], where wanted
  float* sums;
  int32_t blocks;
  int32_t wanted;  // bit q: sum q
};

// The sums over rows.
enum { kDw, kDb, kDgate, kDw1, kDb1, kSums };

// Columns of a thread: 8 for each of V, a 16-byte vector (VEC), or 8 single ones spread
// over the row.  (`lanes` threads share a row.)
template <int V, bool VEC>
struct Columns {
  int at, lanes;
  int64_t width;
  __device__ __forceinline__ int64_t of(int k) const {  // k-th column, 0 to 8 V - 1
    return VEC ? (static_cast<int64_t>(k / 8) * lanes + at) * 8 + k % 8
               : static_cast<int64_t>(k) * lanes + at;
  }
  __device__ __forceinline__ bool in(int k) const { return of(k) < width; }
  // Elements of a row (0 past its end).
  __device__ __forceinline__ void load(const uint16_t* p, float x[8 * V], bool vec = VEC) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (VEC && vec && of(8 * v) + 8 <= width) {
        bf16x8(*reinterpret_cast<const uint4*>(p + of(8 * v)), x + 8 * v);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) x[8 * v + c] = in(8 * v + c) ? bf16_at(p + of(8 * v + c)) : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store(uint16_t* p, const float x[8 * V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (VEC && of(8 * v) + 8 <= width) {
        *reinterpret_cast<uint4*>(p + of(8 * v)) = to_bf16x8(x + 8 * v);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (in(8 * v + c)) p[of(8 * v + c)] = to_bf16(x[8 * v + c]);
      }
    }
  }
  __device__ __forceinline__ void load_or(const uint16_t* p, float x[8 * V], float other, bool vec) const {
    if (p != nullptr) {
      load(p, x, vec);
    } else {
#pragma unroll
      for (int k = 0; k < 8 * V; ++k) x[k] = other;
    }
  }
};

// Sums over the threads of a row: a warp, or a block (through shared memory, in two
// places taken in turn, so that one barrier is enough).
template <bool BLOCK>
struct RowSum {
  float (*part)[kMostThreads / 32][3];
  int place = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float (&x)[N]) {
#pragma unroll
    for (int k = 16; k > 0; k /= 2)
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], k);
    if constexpr (BLOCK) {
      const int warps = blockDim.x / 32;
      if (threadIdx.x % 32 == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) part[place][threadIdx.x / 32][n] = x[n];
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] = 0.0f;
      for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] += part[place][w][n];
      place ^= 1;
    }
  }
};

// x to (x - mean) / root, mean 0 for RMS; columns past the end stay 0.
template <int V, bool VEC, bool BLOCK>
__device__ __forceinline__ void standardize(const Columns<V, VEC>& at, float x[8 * V], bool layer, float eps,
                                            float inv_width, RowSum<BLOCK>& row_sum) {
  if (layer) {
    float m[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < 8 * V; ++k) m[0] += x[k];
    row_sum(m);
    m[0] *= inv_width;
#pragma unroll
    for (int k = 0; k < 8 * V; ++k) x[k] = at.in(k) ? x[k] - m[0] : 0.0f;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < 8 * V; ++k) q[0] = fmaf(x[k], x[k], q[0]);
  row_sum(q);
  const float inverse = rsqrtf(fmaf(q[0], inv_width, eps));
#pragma unroll
  for (int k = 0; k < 8 * V; ++k) x[k] *= inverse;
}

// A row a warp (8 rows a block), or a row a block.
template <int V, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kMostThreads : 256)
    block_norm_forward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][kMostThreads / 32][3];
  wait_for_predecessor();
  launch_dependents();
  constexpr int N = 8 * V;
  const Columns<V, VEC> at{static_cast<int>(BLOCK ? threadIdx.x : threadIdx.x % 32),
                           static_cast<int>(BLOCK ? blockDim.x : 32), a.width};
  RowSum<BLOCK> row_sum{part};
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const bool wvec = a.wvec != 0;
  const int64_t step = BLOCK ? gridDim.x : static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t i = BLOCK ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; i < a.rows;
       i += step) {
    float s[N], t[N];
    at.load(a.r + i * a.ldr, s);
    if (a.h != nullptr) {
      float p[N];
      at.load(a.h + i * a.ldh, p);
      if (a.post != ZERO_NORM_NONE) {
        standardize(at, p, a.post == ZERO_NORM_LAYER, a.eps, inv_width, row_sum);
        if (a.w1 != nullptr) {
          at.load(a.w1, t, wvec);
#pragma unroll
          for (int k = 0; k < N; ++k) p[k] *= t[k];
        }
        if (a.b1 != nullptr) {
          at.load(a.b1, t, wvec);
#pragma unroll
          for (int k = 0; k < N; ++k) p[k] += t[k];
        }
      }
      if (a.gate != nullptr) {
        at.load(a.gate + i * a.ldg, t, a.ldg != 0 || wvec);
#pragma unroll
        for (int k = 0; k < N; ++k) p[k] *= t[k];
      }
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] = fmaf(a.alpha, p[k], s[k]);
    }
    if (a.s_out != nullptr) at.store(a.s_out + i * a.lds, s);
    standardize(at, s, a.kind == ZERO_NORM_LAYER, a.eps, inv_width, row_sum);
    if (a.w != nullptr) {
      at.load(a.w, t, wvec);
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] *= t[k];
    }
    if (a.b != nullptr) {
      at.load(a.b, t, wvec);
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] += t[k];
    }
    at.store(a.y + i * a.ldy, s);
  }
}

// The backward pass: a block takes every gridDim.x-th row, its threads the same columns of
// each, whose sums over the rows stay in their registers until the end.  With xh the
// standardized row, u what reaches it and m its means,
//   x's gradient = (u - m(u) [LAYER] - xh m(u xh)) / root.
// FULL: there is a norm after the block, or a gate: h is read.
template <int V, bool VEC, bool FULL>
__global__ void __launch_bounds__(kMostThreads)
    block_norm_backward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][kMostThreads / 32][3];
  wait_for_predecessor();
  launch_dependents();
  constexpr int N = 8 * V;
  const Columns<V, VEC> at{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.width};
  RowSum<true> row_sum{part};
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const bool wvec = a.wvec != 0;
  const bool layer = a.kind == ZERO_NORM_LAYER, post_layer = a.post == ZERO_NORM_LAYER;
  float dw[N] = {}, db[N] = {}, dg[FULL ? N : 1] = {}, dw1[FULL ? N : 1] = {}, db1[FULL ? N : 1] = {};
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    float x[N], u[N], h[FULL ? N : 1];
    at.load(a.s + i * a.lds, x);
    at.load(a.dy + i * a.lddy, u);
    if constexpr (FULL) at.load(a.h + i * a.ldh, h);
    {
      float w[N];
      at.load_or(a.w, w, 1.0f, wvec);
      // means, then what is left: LAYER
      if (layer || (FULL && post_layer)) {
        float m[3] = {};
#pragma unroll
        for (int k = 0; k < N; ++k) {
          m[0] += x[k];
          if constexpr (FULL) m[1] += h[k];
        }
        row_sum(m);
        if (layer) {
#pragma unroll
          for (int k = 0; k < N; ++k) x[k] = at.in(k) ? x[k] - m[0] * inv_width : 0.0f;
        }
        if constexpr (FULL)
          if (post_layer) {
#pragma unroll
            for (int k = 0; k < N; ++k) h[k] = at.in(k) ? h[k] - m[1] * inv_width : 0.0f;
          }
      }
      float q[3] = {}, su[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < N; ++k) {
        q[0] = fmaf(x[k], x[k], q[0]);
        q[1] = fmaf(u[k] * w[k], x[k], q[1]);
        if constexpr (FULL) q[2] = fmaf(h[k], h[k], q[2]);
        su[0] = fmaf(u[k], w[k], su[0]);
      }
      row_sum(q);
      if (layer) row_sum(su);
      const float inverse = rsqrtf(fmaf(q[0], inv_width, a.eps));
      const float along = q[1] * inverse * inv_width, mean = layer ? su[0] * inv_width : 0.0f;
      if constexpr (FULL) {
        if (a.post != ZERO_NORM_NONE) {
          const float inverse1 = rsqrtf(fmaf(q[2], inv_width, a.eps));
#pragma unroll
          for (int k = 0; k < N; ++k) h[k] *= inverse1;
          q[2] = inverse1;
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float xh = x[k] * inverse;
        dw[k] = fmaf(u[k], xh, dw[k]);
        db[k] += u[k];
        x[k] = at.in(k) ? inverse * (u[k] * w[k] - mean - xh * along) : 0.0f;
      }
      if (a.ds != nullptr) {
        at.load(a.ds + i * a.ldds, u);
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] += u[k];
      }
      if (a.dr != nullptr) at.store(a.dr + i * a.lddr, x);
      if constexpr (!FULL) {
        if (a.dh != nullptr) {
#pragma unroll
          for (int k = 0; k < N; ++k) x[k] *= a.alpha;
          at.store(a.dh + i * a.lddh, x);
        }
      } else {
        // x: the gradient of alpha gate P(h);  h: standardized, or itself
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] *= a.alpha;
        at.load_or(a.w1, w, 1.0f, wvec);
        if (a.gate != nullptr) {
          float g[N];
          at.load_or(a.b1, u, 0.0f, wvec);
          at.load(a.gate + i * a.ldg, g, a.ldg != 0 || wvec);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            u[k] = x[k] * fmaf(h[k], w[k], u[k]);
            dg[k] += u[k];
            x[k] *= g[k];
          }
          if (a.dgate_rows != nullptr) at.store(a.dgate_rows + i * a.lddg, u);
        }
        if (a.post != ZERO_NORM_NONE) {
          float m[2] = {};
#pragma unroll
          for (int k = 0; k < N; ++k) {
            dw1[k] = fmaf(x[k], h[k], dw1[k]);
            db1[k] += x[k];
            x[k] *= w[k];
            m[0] = fmaf(x[k], h[k], m[0]);
            m[1] += x[k];
          }
          if (a.dh != nullptr) {  // (alike for every thread)
            row_sum(m);
            m[0] *= inv_width;
            m[1] = post_layer ? m[1] * inv_width : 0.0f;
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = q[2] * (x[k] - m[1] - h[k] * m[0]);
          }
        }
        if (a.dh != nullptr) at.store(a.dh + i * a.lddh, x);
      }
    }
  }
  const auto put = [&](int q, const float* x) {
    if ((a.wanted >> q & 1) == 0) return;
    float* to = a.sums + (static_cast<int64_t>(q) * a.blocks + blockIdx.x) * a.width;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at.in(k)) to[at.of(k)] = x[k];
  };
  put(kDw, dw);
  put(kDb, db);
  if constexpr (FULL) {
    put(kDgate, dg);
    put(kDw1, dw1);
    put(kDb1, db1);
  }
}

struct NormJoinArgs {
  const float* sums;
  int64_t width;
  int32_t blocks;  // 0: sums of nothing
  void* out[kSums];
  int32_t out_f32, accumulate;
};

// The blocks' sums in their order: 32 columns a block, 8 runs of blocks, which are added
// up in their order too.
__global__ void __launch_bounds__(256) block_norm_join_kernel(const __grid_constant__ NormJoinArgs a) {
  __shared__ float part[8][33];
  wait_for_predecessor();
  launch_dependents();
  void* out = a.out[blockIdx.y];
  if (out == nullptr) return;
  const int r = threadIdx.x / 32, c = threadIdx.x % 32;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float sum = 0.0f;
  if (j < a.width) {
    const float* p = a.sums + static_cast<int64_t>(blockIdx.y) * a.blocks * a.width + j;
#pragma unroll 8
    for (int k = r; k < a.blocks; k += 8) sum += __ldcg(p + k * a.width);
  }
  part[r][c] = sum;
  __syncthreads();
  if (r != 0 || j >= a.width) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) sum += part[k][c];
  if (a.out_f32) {
    float* o = static_cast<float*>(out) + j;
    *o = a.accumulate ? *o + sum : sum;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + j;
    *o = to_bf16(a.accumulate ? bf16_at(o) + sum : sum);
  }
}

// Blocks of the backward pass: 4 rows each at least, two blocks an SM at most.
int64_t backward_blocks(int64_t rows) {
  const int64_t n = (rows + 3) / 4;
  return n < 2 * kSms ? n : 2 * kSms;
}

NormArgs args_of(const BlockNormLaunch& L) {
  const zero_block_norm_t& s = L.s;
  NormArgs a{};
  a.rows = s.rows;
  a.width = s.width;
  a.post = L.h != nullptr ? s.post : ZERO_NORM_NONE;
  a.kind = s.kind;
  a.alpha = static_cast<float>(s.alpha);
  a.eps = static_cast<float>(s.eps);
  a.r = L.r; a.h = L.h; a.w1 = L.post_weight; a.b1 = L.post_bias; a.gate = L.gate;
  a.w = L.weight; a.b = L.bias; a.s_out = L.s_out; a.y = L.y;
  a.dy = L.dy; a.ds = L.ds; a.s = L.sum; a.dr = L.dr; a.dh = L.dh;
  a.ldr = s.ldr; a.ldh = s.ldh; a.ldg = s.ldg; a.lds = s.lds; a.ldy = s.ldy;
  a.lddy = s.lddy; a.ldds = s.ldds; a.lddr = s.lddr; a.lddh = s.lddh; a.lddg = s.lddg;
  a.wvec = 1;
  for (const void* p : {static_cast<const void*>(L.post_weight), static_cast<const void*>(L.post_bias),
                        static_cast<const void*>(L.weight), static_cast<const void*>(L.bias),
                        static_cast<const void*>(s.ldg == 0 ? L.gate : nullptr)})
    if (!aligned(p, 16)) a.wvec = 0;
  return a;
}

// Whether rows of every matrix lie on 16-byte boundaries.
struct Rows16 {
  int64_t rows;
  bool all = true;
  void operator()(const void* p, int64_t ld) {
    if (p != nullptr && (!aligned(p, 16) || (rows > 1 && ld % 8 != 0))) all = false;
  }
};

template <bool VEC, bool FULL>
cudaError_t launch_backward(const NormArgs& a, int vectors, int threads, Chain* chain) {
  const auto kernel = vectors <= 1   ? block_norm_backward_kernel<1, VEC, FULL>
                      : vectors <= 2 ? block_norm_backward_kernel<2, VEC, FULL>
                      : vectors <= 4 ? block_norm_backward_kernel<4, VEC, FULL>
                                     : block_norm_backward_kernel<8, VEC, FULL>;
  return chain->launch(kernel, dim3(a.blocks), threads, 0, 1, a);
}

template <bool VEC>
cudaError_t launch_forward(const NormArgs& a, Chain* chain) {
  const int64_t eights = (a.width + 7) / 8;
  // a warp a row up to 1,024 columns (no barriers), else a block
  if (eights <= 128) {
    const int64_t blocks = (a.rows + 7) / 8;
    const auto kernel = eights <= 32   ? block_norm_forward_kernel<1, VEC, false>
                        : eights <= 64 ? block_norm_forward_kernel<2, VEC, false>
                                       : block_norm_forward_kernel<4, VEC, false>;
    return chain->launch(kernel, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), 256, 0, 1, a);
  }
  const int64_t warps = (eights + 31) / 32;
  const int threads = static_cast<int>(32 * warps < kMostThreads ? 32 * warps : kMostThreads);
  const int64_t vectors = (eights + threads - 1) / threads;
  const auto kernel = vectors <= 1   ? block_norm_forward_kernel<1, VEC, true>
                      : vectors <= 2 ? block_norm_forward_kernel<2, VEC, true>
                      : vectors <= 4 ? block_norm_forward_kernel<4, VEC, true>
                                     : block_norm_forward_kernel<8, VEC, true>;
  return chain->launch(kernel, dim3(static_cast<unsigned>(a.rows < 65536 ? a.rows : 65536)), threads, 0, 1, a);
}

}  // namespace

int64_t block_norm_workspace(const zero_block_norm_t& s) {
  return round_up(4 * kSums * backward_blocks(s.rows) * s.width, 256);
}

cudaError_t launch_block_norm_forward(const BlockNormLaunch& L) {
  (void)cudaGetLastError();
  const NormArgs a = args_of(L);
  Rows16 vec{a.rows};
  vec(a.r, a.ldr);
  vec(a.h, a.ldh);
  vec(a.s_out, a.lds);
  vec(a.y, a.ldy);
  if (a.ldg != 0) vec(a.gate, a.ldg);
  Chain chain{L.stream};
  return vec.all ? launch_forward<true>(a, &chain) : launch_forward<false>(a, &chain);
}

cudaError_t launch_block_norm_backward(const BlockNormLaunch& L) {
  (void)cudaGetLastError();
  NormArgs a = args_of(L);
  NormJoinArgs j{};
  j.out[kDw] = L.dweight;
  j.out[kDb] = L.dbias;
  j.out[kDgate] = a.ldg == 0 ? L.dgate : nullptr;
  j.out[kDw1] = L.dpost_weight;
  j.out[kDb1] = L.dpost_bias;
  a.dgate_rows = a.ldg != 0 ? static_cast<uint16_t*>(L.dgate) : nullptr;
  for (int q = 0; q < kSums; ++q) a.wanted |= (j.out[q] != nullptr ? 1 : 0) << q;
  Chain chain{L.stream};
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    Rows16 vec{a.rows};
    vec(a.dy, a.lddy);
    vec(a.ds, a.ldds);
    vec(a.s, a.lds);
    vec(a.h, a.ldh);
    vec(a.dr, a.lddr);
    vec(a.dh, a.lddh);
    if (a.ldg != 0) {
      vec(a.gate, a.ldg);
      vec(a.dgate_rows, a.lddg);
    }
    a.sums = static_cast<float*>(L.workspace);
    a.blocks = static_cast<int32_t>(backward_blocks(a.rows));
    const bool full = a.h != nullptr && (a.post != ZERO_NORM_NONE || a.gate != nullptr);
    const int64_t eights = (a.width + 7) / 8, warps = (eights + 31) / 32;
    const int threads = static_cast<int>(32 * warps < kMostThreads ? 32 * warps : kMostThreads);
    const int vectors = static_cast<int>((eights + threads - 1) / threads);
    e = vec.all ? (full ? launch_backward<true, true>(a, vectors, threads, &chain)
                        : launch_backward<true, false>(a, vectors, threads, &chain))
                : (full ? launch_backward<false, true>(a, vectors, threads, &chain)
                        : launch_backward<false, false>(a, vectors, threads, &chain));
  }
  if (e != cudaSuccess || a.wanted == 0 || (a.rows == 0 && L.accumulate)) return e;
  j.sums = a.sums;
  j.width = a.width;
  j.blocks = a.rows > 0 ? a.blocks : 0;
  j.out_f32 = L.grad_f32;
  j.accumulate = L.accumulate;
  return chain.launch(block_norm_join_kernel, dim3(static_cast<unsigned>((a.width + 31) / 32), kSums), 256, 0,
                      1, j);
}

}  // namespace zeroadam
