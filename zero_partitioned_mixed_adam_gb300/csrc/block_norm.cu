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

constexpr int kMostThreads = 512, kMostWarps = kMostThreads / 32, kMostCluster = 8;
constexpr int kStages = 4;  // rows under way

// Who shares a row: a warp up to 1,024 columns (forward), a block up to 4,096, a cluster of
// blocks beyond.  A thread's columns are few in every case, so that the backward pass has
// room for the sums of each in registers.
enum Share { kWarp, kBlock, kCluster };

__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

// What a row is read from.
enum Input { kInR, kInH, kInGate, kInDy, kInDs, kInputs };

struct NormArgs {
  int64_t rows, width;
  int32_t post, kind;
  float alpha, eps;
  const uint16_t* in[kInputs];  // NULL: not there (kInR is the backward pass's s)
  int64_t ld[kInputs];
  int32_t place[kInputs];       // in a stage of the ring
  int32_t inputs;
  const uint16_t *gate, *w1, *b1, *w, *b;  // vectors (gate: or NULL, kInGate is a matrix)
  uint16_t *s_out, *y;
  uint16_t *dr, *dh, *dgate_rows;          // dgate_rows: a matrix
  int64_t lds, ldy, lddr, lddh, lddg;
  int32_t wvec;    // the vectors are read 16 bytes at a time
  // backward: sums of each block's rows, [kSums][blocks][width], where wanted
  float* sums;
  int32_t blocks;
  int32_t wanted;  // bit q: sum q
};

// The sums over rows.
enum { kDw, kDgate, kDw1, kDb, kDb1, kSums };

__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Columns of a thread: 8 for each of V, a 16-byte vector (VEC), or 8 single ones spread
// over the row.  (`lanes` threads share a row.)
template <int V, bool VEC>
struct Columns {
  int at, lanes;
  int width;
  __device__ __forceinline__ int of(int k) const {  // k-th column, 0 to 8 V - 1
    return VEC ? (k / 8 * lanes + at) * 8 + k % 8 : k * lanes + at;
  }
  __device__ __forceinline__ bool in(int k) const { return of(k) < width; }
  __device__ __forceinline__ bool whole(int v) const { return VEC && of(8 * v) + 8 <= width; }
  // Elements of a row (0 past its end).
  __device__ __forceinline__ void load(const uint16_t* p, float x[8 * V], bool vec = VEC) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (vec && whole(v)) {
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
      if (whole(v)) {
        *reinterpret_cast<uint4*>(p + of(8 * v)) = to_bf16x8(x + 8 * v);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (in(8 * v + c)) p[of(8 * v + c)] = to_bf16(x[8 * v + c]);
      }
    }
  }
};

// A vector of the columns, held in registers as bf16: 4 of them for 8 columns.
template <int V>
struct Held {
  uint32_t p[4 * V];
  template <bool VEC>
  __device__ __forceinline__ Held(const Columns<V, VEC>& at, const uint16_t* from, float other, bool vec) {
    float x[8 * V];
    if (from != nullptr) at.load(from, x, vec);
#pragma unroll
    for (int k = 0; k < 4 * V; ++k)
      p[k] = from != nullptr ? bf16x2_bits(x[2 * k], x[2 * k + 1]) : bf16x2_bits(other, other);
  }
  __device__ __forceinline__ float operator[](int k) const {
    return __uint_as_float(k % 2 ? p[k / 2] & 0xffff0000u : p[k / 2] << 16);
  }
};

// The rows that a thread reads, kStages ahead (RING): its own 16 bytes of each input, from
// its own place in shared memory, so no thread waits for another's.  Rows that are not on
// 16-byte boundaries, and those too wide for the ring, are read when they are wanted.
template <int V, bool VEC, bool RING>
struct Rows {
  const NormArgs& a;
  const Columns<V, VEC>& at;
  uint8_t* ring;      // of this thread
  int32_t threads;    // of the block
  int64_t next;       // the row that is asked for next
  int64_t step;
  int put = 0, got = 0;

  __device__ __forceinline__ uint8_t* slot(int stage, int q, int v) const {
    return ring + ((stage * a.inputs + a.place[q]) * V + v) * threads * 16;
  }
  __device__ __forceinline__ void ask() {
    if constexpr (RING) {
      if (next < a.rows) {
#pragma unroll
        for (int q = 0; q < kInputs; ++q) {
          if (a.in[q] == nullptr) continue;
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (at.whole(v)) copy16(slot(put, q, v), a.in[q] + next * a.ld[q] + at.of(8 * v));
        }
      }
      next += step;
      put = put + 1 == kStages ? 0 : put + 1;
      copy_commit();
    }
  }
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int k = 1; k < kStages; ++k) ask();
  }
  // The row after the last can be read.
  __device__ __forceinline__ void arrive() {
    if constexpr (RING) {
      ask();
      copy_wait<kStages - 1>();
    }
  }
  __device__ __forceinline__ void read(int q, int64_t i, float x[8 * V]) const {
    if constexpr (RING) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (at.whole(v)) {
          bf16x8(*reinterpret_cast<const uint4*>(slot(got, q, v)), x + 8 * v);
        } else {
          const uint16_t* p = a.in[q] + i * a.ld[q];
#pragma unroll
          for (int c = 0; c < 8; ++c) x[8 * v + c] = at.in(8 * v + c) ? bf16_at(p + at.of(8 * v + c)) : 0.0f;
        }
      }
    } else {
      at.load(a.in[q] + i * a.ld[q], x);
    }
  }
  __device__ __forceinline__ void done() { got = got + 1 == kStages ? 0 : got + 1; }
};

// Sums over the threads of a row, in the same order for each of them.  The warps' parts go
// through shared memory, every block's to all blocks of the cluster, in two places taken in
// turn, so that one barrier is enough: a place is written again only after the barrier
// that follows its reading.
template <Share SHARE>
struct RowSum {
  static constexpr int kParts = SHARE == kWarp ? 1 : SHARE == kBlock ? kMostWarps : kMostCluster * kMostWarps;
  float4 (*part)[kParts];
  int place = 0;
  __device__ __forceinline__ float3 operator()(float x, float y = 0.0f, float z = 0.0f) {
    const auto add_lanes = [&] {
#pragma unroll
      for (int k = 16; k > 0; k /= 2) {
        x += __shfl_xor_sync(0xffffffffu, x, k);
        y += __shfl_xor_sync(0xffffffffu, y, k);
        z += __shfl_xor_sync(0xffffffffu, z, k);
      }
    };
    add_lanes();
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if constexpr (SHARE == kBlock) {
      if (lane == 0) part[place][warp] = make_float4(x, y, z, 0.0f);
      __syncthreads();
      x = y = z = 0.0f;
#pragma unroll 4
      for (int w = 0; w < warps; ++w) {
        const float4 p = part[place][w];
        x += p.x;
        y += p.y;
        z += p.z;
      }
      place ^= 1;
    } else if constexpr (SHARE == kCluster) {
      const int blocks = static_cast<int>(cluster_blocks());
      if (lane < blocks)
        peer_store(peer_addr(&part[place][static_cast<int>(cluster_rank()) * warps + warp], lane),
                   make_float4(x, y, z, 0.0f));
      cluster_sync_writes();
      x = y = z = 0.0f;
      for (int w = lane; w < blocks * warps; w += 32) {
        const float4 p = part[place][w];
        x += p.x;
        y += p.y;
        z += p.z;
      }
      add_lanes();
      place ^= 1;
    }
    return make_float3(x, y, z);
  }
};

// A row's threads, and which rows they take.
template <Share SHARE>
struct RowOwner {
  int at, lanes;        // this thread's place among the row's
  int64_t first, step;  // rows
  __device__ __forceinline__ RowOwner() {
    if constexpr (SHARE == kWarp) {
      at = threadIdx.x % 32;
      lanes = 32;
      first = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
      step = static_cast<int64_t>(gridDim.x) * 8;
    } else if constexpr (SHARE == kBlock) {
      at = threadIdx.x;
      lanes = blockDim.x;
      first = blockIdx.x;
      step = gridDim.x;
    } else {
      const int blocks = static_cast<int>(cluster_blocks());
      at = static_cast<int>(cluster_rank() * blockDim.x + threadIdx.x);
      lanes = blocks * blockDim.x;
      first = blockIdx.x / blocks;
      step = gridDim.x / blocks;
    }
  }
};

// x to (x - mean) / root, mean 0 for RMS; columns past the end stay 0.
template <int V, bool VEC, Share SHARE>
__device__ __forceinline__ void standardize(const Columns<V, VEC>& at, float x[8 * V], bool layer, float eps,
                                            float inv_width, RowSum<SHARE>& row_sum) {
  if (layer) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8 * V; ++k) m += x[k];
    m = row_sum(m).x * inv_width;
#pragma unroll
    for (int k = 0; k < 8 * V; ++k) x[k] = at.in(k) ? x[k] - m : 0.0f;
  }
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < 8 * V; ++k) q = fmaf(x[k], x[k], q);
  const float inverse = rsqrtf(fmaf(row_sum(q).x, inv_width, eps));
#pragma unroll
  for (int k = 0; k < 8 * V; ++k) x[k] *= inverse;
}

template <int V, bool VEC, Share SHARE, bool RING>
__global__ void __launch_bounds__(SHARE == kWarp ? 256 : kMostThreads)
    block_norm_forward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float4 part[2][RowSum<SHARE>::kParts];
  extern __shared__ uint8_t ring[];
  wait_for_predecessor();
  launch_dependents();
  constexpr int N = 8 * V;
  const RowOwner<SHARE> own;
  const Columns<V, VEC> at{own.at, own.lanes, static_cast<int>(a.width)};
  RowSum<SHARE> row_sum{part};
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const bool wvec = a.wvec != 0;
  Rows<V, VEC, RING> rows{a, at, ring + threadIdx.x * 16, static_cast<int32_t>(blockDim.x), own.first, own.step};
  rows.begin();
  for (int64_t i = own.first; i < a.rows; i += own.step, rows.done()) {
    float s[N], t[N];
    rows.arrive();
    rows.read(kInR, i, s);
    if (a.in[kInH] != nullptr) {
      float p[N];
      rows.read(kInH, i, p);
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
      const bool matrix = a.in[kInGate] != nullptr;
      if (matrix || a.gate != nullptr) {
        if (matrix) rows.read(kInGate, i, t);
        else at.load(a.gate, t, wvec);
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
  if constexpr (SHARE == kCluster) cluster_sync();  // no block ends while others write to it
}

// The backward pass: a block (or cluster) takes every so-many-th row, its threads the same 8
// columns of each, whose sums over the rows stay in their registers until the end.  With xh
// the standardized row, u what reaches it and m its means,
//   x's gradient = (u - m(u) [LAYER] - xh m(u xh)) / root.
// FULL: there is a norm after the block, or a gate: h is read.  BIAS: sums of biases.
template <bool VEC, Share SHARE, bool FULL, bool BIAS>
__global__ void __launch_bounds__(kMostThreads)
    block_norm_backward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float4 part[2][RowSum<SHARE>::kParts];
  extern __shared__ uint8_t ring[];
  wait_for_predecessor();
  launch_dependents();
  constexpr int N = 8, M = FULL ? N : 1;
  const RowOwner<SHARE> own;
  const Columns<1, VEC> at{own.at, own.lanes, static_cast<int>(a.width)};
  RowSum<SHARE> row_sum{part};
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const bool wvec = a.wvec != 0;
  const bool layer = a.kind == ZERO_NORM_LAYER, post_layer = a.post == ZERO_NORM_LAYER;
  const bool post = a.post != ZERO_NORM_NONE;
  const Held<1> w(at, a.w, 1.0f, wvec);
  float dw[N] = {}, db[BIAS ? N : 1] = {}, dg[M] = {}, dw1[M] = {}, db1[BIAS ? M : 1] = {};
  Rows<1, VEC, VEC> rows{a, at, ring + threadIdx.x * 16, static_cast<int32_t>(blockDim.x), own.first, own.step};
  rows.begin();
  for (int64_t i = own.first; i < a.rows; i += own.step, rows.done()) {
    float x[N], u[N], h[M];
    rows.arrive();
    rows.read(kInR, i, x);
    rows.read(kInDy, i, u);
    if constexpr (FULL) rows.read(kInH, i, h);
    if (layer || (FULL && post_layer)) {  // means, then what is left
      float m = 0.0f, m1 = 0.0f;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        m += x[k];
        if constexpr (FULL) m1 += h[k];
      }
      const float3 means = row_sum(m, m1);
      if (layer) {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = at.in(k) ? x[k] - means.x * inv_width : 0.0f;
      }
      if constexpr (FULL)
        if (post_layer) {
#pragma unroll
          for (int k = 0; k < N; ++k) h[k] = at.in(k) ? h[k] - means.y * inv_width : 0.0f;
        }
    }
    float xx = 0.0f, ux = 0.0f, hh = 0.0f, mean = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      xx = fmaf(x[k], x[k], xx);
      ux = fmaf(u[k] * w[k], x[k], ux);
      if constexpr (FULL) hh = fmaf(h[k], h[k], hh);
    }
    if (layer) {
#pragma unroll
      for (int k = 0; k < N; ++k) mean = fmaf(u[k], w[k], mean);
      mean = row_sum(mean).x * inv_width;
    }
    const float3 q = row_sum(xx, ux, hh);
    const float inverse = rsqrtf(fmaf(q.x, inv_width, a.eps));
    const float along = q.y * inverse * inv_width;
    const float inverse1 = FULL && post ? rsqrtf(fmaf(q.z, inv_width, a.eps)) : 1.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float xh = x[k] * inverse;
      dw[k] = fmaf(u[k], xh, dw[k]);
      if constexpr (BIAS) db[k] += u[k];
      x[k] = at.in(k) ? inverse * (u[k] * w[k] - mean - xh * along) : 0.0f;
    }
    if (a.in[kInDs] != nullptr) {
      rows.read(kInDs, i, u);
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] += u[k];
    }
    if (a.dr != nullptr) at.store(a.dr + i * a.lddr, x);
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] *= a.alpha;  // the gradient of gate P(h)
    if constexpr (!FULL) {
      if (a.dh != nullptr) at.store(a.dh + i * a.lddh, x);
    } else {
      float w1[N], g[N];
      if (post) {
#pragma unroll
        for (int k = 0; k < N; ++k) h[k] *= inverse1;  // standardized
      }
      if (a.w1 != nullptr) {
        at.load(a.w1, w1, wvec);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) w1[k] = 1.0f;
      }
      const bool matrix = a.in[kInGate] != nullptr;
      if (matrix || a.gate != nullptr) {
        if (a.b1 != nullptr) {
          at.load(a.b1, u, wvec);
        } else {
#pragma unroll
          for (int k = 0; k < N; ++k) u[k] = 0.0f;
        }
        if (matrix) rows.read(kInGate, i, g);
        else at.load(a.gate, g, wvec);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          u[k] = x[k] * fmaf(h[k], w1[k], u[k]);
          dg[k] += u[k];
          x[k] *= g[k];
        }
        if (a.dgate_rows != nullptr) at.store(a.dgate_rows + i * a.lddg, u);
      }
      if (post) {
        float vh = 0.0f, v = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          dw1[k] = fmaf(x[k], h[k], dw1[k]);
          if constexpr (BIAS) db1[k] += x[k];
          x[k] *= w1[k];
          vh = fmaf(x[k], h[k], vh);
          v += x[k];
        }
        if (a.dh != nullptr) {  // (alike for every thread)
          const float3 m = row_sum(vh, v);
          const float along1 = m.x * inv_width, mean1 = post_layer ? m.y * inv_width : 0.0f;
#pragma unroll
          for (int k = 0; k < N; ++k) x[k] = inverse1 * (x[k] - mean1 - h[k] * along1);
        }
      }
      if (a.dh != nullptr) at.store(a.dh + i * a.lddh, x);
    }
  }
  const auto put = [&](int q, const float* x) {
    if ((a.wanted >> q & 1) == 0) return;
    float* to = a.sums + (static_cast<int64_t>(q) * a.blocks + own.first) * a.width;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at.in(k)) to[at.of(k)] = x[k];
  };
  put(kDw, dw);
  if constexpr (BIAS) put(kDb, db);
  if constexpr (FULL) {
    put(kDgate, dg);
    put(kDw1, dw1);
    if constexpr (BIAS) put(kDb1, db1);
  }
  if constexpr (SHARE == kCluster) cluster_sync();  // no block ends while others write to it
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

// Blocks that share a row, and threads of each: 8 columns a thread.
struct RowShape {
  int cluster, threads;
};
RowShape row_shape(int64_t width) {
  const int64_t eights = (width + 7) / 8;
  int cluster = 1;
  while (eights > cluster * kMostThreads) cluster *= 2;
  return {cluster, static_cast<int>(round_up((eights + cluster - 1) / cluster, 32))};
}
static_assert(ZERO_MAX_NORM_WIDTH == 8 * kMostThreads * kMostCluster, "the widest row's cluster");

// Blocks (clusters) of the backward pass: 4 rows each at least, and as many as are there at
// one time (768 threads an SM).
int64_t backward_blocks(int64_t rows, int64_t width) {
  const RowShape r = row_shape(width);
  const int64_t n = (rows + 3) / 4;
  const int64_t most = kSms / r.cluster * (r.threads < 64 ? 12 : 768 / r.threads);
  return n < most ? n : most;
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
  a.w1 = L.post_weight;
  a.b1 = L.post_bias;
  a.w = L.weight;
  a.b = L.bias;
  (s.ldg == 0 ? a.gate : a.in[kInGate]) = L.gate;
  a.ld[kInGate] = s.ldg;
  a.in[kInH] = L.h;
  a.ld[kInH] = s.ldh;
  a.s_out = L.s_out;
  a.y = L.y;
  a.dr = L.dr;
  a.dh = L.dh;
  a.lds = s.lds;
  a.ldy = s.ldy;
  a.lddr = s.lddr;
  a.lddh = s.lddh;
  a.lddg = s.lddg;
  a.wvec = 1;
  for (const uint16_t* p : {a.w1, a.b1, a.w, a.b, a.gate})
    if (!aligned(p, 16)) a.wvec = 0;
  return a;
}

// Bytes of the ring, for each thread 16 of each vector of each input.
constexpr int kMostRing = kStages * kInputs * kMostThreads * 16;
static_assert(kMostRing + 8192 <= kSmem, "the ring and the parts of the sums");
int ring_bytes(const NormArgs& a, int vectors, int threads) {
  return kStages * a.inputs * vectors * threads * 16;
}

// Whether rows of every matrix lie on 16-byte boundaries; and the inputs' places.
struct Rows16 {
  int64_t rows;
  bool all = true;
  void operator()(const void* p, int64_t ld) {
    if (p != nullptr && (!aligned(p, 16) || (rows > 1 && ld % 8 != 0))) all = false;
  }
  explicit Rows16(NormArgs* a) : rows(a->rows) {
    for (int q = 0; q < kInputs; ++q) {
      (*this)(a->in[q], a->ld[q]);
      if (a->in[q] != nullptr) a->place[q] = a->inputs++;
    }
  }
};

// A kernel with a ring of `smem` bytes.
template <typename Kernel>
cudaError_t launch_ring(Kernel kernel, int64_t blocks, int threads, int smem, int cluster, const NormArgs& a,
                        Chain* chain) {
  if (smem > 40 * 1024) {
    // (a property of the kernel on the current device, set alike by every call)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing);
    if (e != cudaSuccess) return e;
  }
  return chain->launch(kernel, dim3(static_cast<unsigned>(blocks * cluster)), threads, smem, cluster, a);
}

template <bool FULL, bool BIAS>
cudaError_t launch_backward(const NormArgs& a, bool vec, Chain* chain) {
  const RowShape r = row_shape(a.width);
  const auto kernel = vec ? (r.cluster == 1 ? block_norm_backward_kernel<true, kBlock, FULL, BIAS>
                                            : block_norm_backward_kernel<true, kCluster, FULL, BIAS>)
                          : (r.cluster == 1 ? block_norm_backward_kernel<false, kBlock, FULL, BIAS>
                                            : block_norm_backward_kernel<false, kCluster, FULL, BIAS>);
  return launch_ring(kernel, a.blocks, r.threads, vec ? ring_bytes(a, 1, r.threads) : 0, r.cluster, a, chain);
}

cudaError_t launch_forward(const NormArgs& a, bool vec, Chain* chain) {
  const int64_t eights = (a.width + 7) / 8;
  if (eights <= 128 && a.rows >= 8 * kSms) {  // (of fewer rows each is made by more threads)
    const int v = static_cast<int>((eights + 31) / 32);
    const int64_t blocks = (a.rows + 7) / 8;
    const int smem = ring_bytes(a, v, 256);
    if (vec && v <= 2)
      return launch_ring(v == 1 ? block_norm_forward_kernel<1, true, kWarp, true>
                                : block_norm_forward_kernel<2, true, kWarp, true>,
                         blocks < 4 * kSms ? blocks : 4 * kSms, 256, smem, 1, a, chain);
    const auto kernel = vec ? (v == 3 ? block_norm_forward_kernel<3, true, kWarp, false>
                                      : block_norm_forward_kernel<4, true, kWarp, false>)
                            : (v <= 2 ? block_norm_forward_kernel<2, false, kWarp, false>
                                      : block_norm_forward_kernel<4, false, kWarp, false>);
    return launch_ring(kernel, blocks < 65536 ? blocks : 65536, 256, 0, 1, a, chain);
  }
  const RowShape r = row_shape(a.width);
  const int smem = vec ? ring_bytes(a, 1, r.threads) : 0;
  int64_t each = 2048 / r.threads;  // blocks an SM
  if (each > 16) each = 16;
  if (each > kSmem / (smem + 1536)) each = kSmem / (smem + 1536);
  const int64_t most = each * kSms / r.cluster;
  const auto kernel = vec ? (r.cluster == 1 ? block_norm_forward_kernel<1, true, kBlock, true>
                                            : block_norm_forward_kernel<1, true, kCluster, true>)
                          : (r.cluster == 1 ? block_norm_forward_kernel<1, false, kBlock, false>
                                            : block_norm_forward_kernel<1, false, kCluster, false>);
  return launch_ring(kernel, a.rows < most ? a.rows : most, r.threads, smem, r.cluster, a, chain);
}

}  // namespace

int64_t block_norm_workspace(const zero_block_norm_t& s) {
  return round_up(4 * kSums * backward_blocks(s.rows, s.width) * s.width, 256);
}

cudaError_t launch_block_norm_forward(const BlockNormLaunch& L) {
  (void)cudaGetLastError();
  NormArgs a = args_of(L);
  a.in[kInR] = L.r;
  a.ld[kInR] = L.s.ldr;
  Rows16 vec(&a);
  vec(a.s_out, a.lds);
  vec(a.y, a.ldy);
  Chain chain{L.stream};
  return launch_forward(a, vec.all, &chain);
}

cudaError_t launch_block_norm_backward(const BlockNormLaunch& L) {
  (void)cudaGetLastError();
  NormArgs a = args_of(L);
  const bool one = L.s.ldg == 0;
  a.in[kInR] = L.sum;
  a.ld[kInR] = L.s.lds;
  a.in[kInDy] = L.dy;
  a.ld[kInDy] = L.s.lddy;
  a.in[kInDs] = L.ds;
  a.ld[kInDs] = L.s.ldds;
  const bool full = L.h != nullptr && (a.post != ZERO_NORM_NONE || L.gate != nullptr);
  if (!full) a.in[kInH] = nullptr;  // (its values are not needed)
  NormJoinArgs j{};
  j.out[kDw] = L.dweight;
  j.out[kDb] = L.dbias;
  j.out[kDgate] = one ? L.dgate : nullptr;
  j.out[kDw1] = L.dpost_weight;
  j.out[kDb1] = L.dpost_bias;
  a.dgate_rows = one ? nullptr : static_cast<uint16_t*>(L.dgate);
  for (int q = 0; q < kSums; ++q) a.wanted |= (j.out[q] != nullptr ? 1 : 0) << q;
  Chain chain{L.stream};
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    Rows16 vec(&a);
    vec(a.dr, a.lddr);
    vec(a.dh, a.lddh);
    vec(a.dgate_rows, a.lddg);
    a.sums = static_cast<float*>(L.workspace);
    a.blocks = static_cast<int32_t>(backward_blocks(a.rows, a.width));
    const bool bias = L.dbias != nullptr || L.dpost_bias != nullptr;
    e = full ? (bias ? launch_backward<true, true>(a, vec.all, &chain)
                     : launch_backward<true, false>(a, vec.all, &chain))
             : (bias ? launch_backward<false, true>(a, vec.all, &chain)
                     : launch_backward<false, false>(a, vec.all, &chain));
  }
  if (e != cudaSuccess || a.wanted == 0 || (a.rows == 0 && L.accumulate)) return e;
  j.sums = a.sums;
  j.width = a.width;
  j.blocks = a.rows > 0 ? a.blocks : 0;
  j.out_f32 = L.grad_f32;
  j.accumulate = L.accumulate;
  // the sums of biases are the last ones
  const unsigned kinds = L.dbias != nullptr || L.dpost_bias != nullptr ? kSums : kDb;
  return chain.launch(block_norm_join_kernel, dim3(static_cast<unsigned>((a.width + 31) / 32), kinds), 256, 0, 1,
                      j);
}

}  // namespace zeroadam
