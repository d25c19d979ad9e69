// cross_entropy.cu -- softmax cross entropy of a linear map onto a vocabulary, and
// its gradients, on sm_103a.
//
// With z = x W^T, a row's loss is log(sum over j of exp(z_j)) - z_t.  z is never kept.
// A row's exponentials are taken less a reference r that is there before the product:
// the target's logit z_t itself, one dot product a row.  Then, S' the sum over j != t,
//   loss = log(1 + S'),   p_j = exp(z_j - z_t) / (1 + S'),   1 - p_t = S' / (1 + S'),
// where nothing is lost to cancellation however sure the model is.  The gradient of z is
// dz_j = c (p_j - [j = t]) = f e_j with one f = c / (1 + S') a row, e_j = exp(z_j - z_t), and
// e_t = -S'.  The product's epilogue writes e in bf16, whose exponent has room for all of it, and
// adds up S'; then dx_i = f_i sum over j of e_ij W_j takes f in its epilogue, and
// dw_j = sum over i of e_ij (f_i x_i) takes x with f in it, rounded to bf16.  So nothing passes over
// the [rows][vocab] values between the products, which read them as they were written (with a
// pass that makes dz of them in place 8192 x 2048 -> 50257 took 3,400 us instead of 3,100, and
// 4096 x 768 -> 50257 709 instead of 600).  The price is one more rounding in dw, of f x: for a
// token that is the target of many rows it averages out (these two cases' dw is 1.05 times as
// far from the exact one as its own rounding puts it), for those of one row it does not (1.4
// times).  So where the values stay in L2, up to 2^25 of them, that pass is made, and dz is
// rounded to bf16 there (1.0 to 1.4 times, of 3 columns up to 1.7).
// A row whose S' passes 2^64 (the target 44 below the largest logit) leaves the range where
// products with 1 / S' lose nothing: its reference becomes the largest logit, which the first
// product found, and product and ends run once more; the launches that do so end at once
// where no row needs them.
//
// Kernels of one piece of rows:
//   places    which rows are not ignored: only they take part in what follows
//   rows      z_t, the reference, the target as a column, x where TMA can read it
//   product   (linear.cu) e and its sums
//   ends      losses, e_t, f, f x (or dz);  product and ends again, where some row needs it
//   products  (linear.cu) dx, dw
//   spread    dx where the caller's rows are
// Small problems leave out places and spread, as their launches are worth more than the rows.
// The loss alone needs neither reference nor x laid out: its product takes the exponentials
// less the largest logit so far, and a warp a row ends it.  The target's logit is a dot
// product of its own there too, rounded to nearest: the tensor cores cut off, and what
// that takes from one logit of 12 is 10 times the loss's other errors.
#include <type_traits>

#include "chain.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

constexpr int64_t kMostHeld = int64_t{1} << 30;  // bytes of e of one piece
constexpr float kOneMore = 18446744073709551616.0f;  // 2^64: a sum that asks for another reference

// Words of the workspace that a call's kernels share.
struct Words {
  int32_t ticket;  // blocks of a kernel that are done
  int32_t again;   // some row of this piece wants another reference
  int32_t rows;    // that are not ignored, of this piece
  float share;     // 1 / rows that are not ignored: c of the mean (0 where there is none)
};

struct LossArgs {
  const uint16_t *x, *w;
  int64_t ldx, ldw;
  const void* targets;
  int32_t ids_i32;
  int64_t ignore;
  int64_t all_rows;       // of all pieces
  int64_t first, rows;    // of this piece
  int64_t width, vocab;
  Words* words;
  float *zt, *ref;        // [rows]
  int32_t* column;        // [rows]; -1: ignored, -2: not a column
  uint16_t* xc;           // [rows][ldxc]
  int64_t ldxc;
  const float2* sums;     // [rows][parts]
  int32_t parts;
  const float* scale;     // [all_rows] or NULL
  float* losses;          // [all_rows]
  float* total;           // NULL: not wanted, or this is not the last piece
  uint16_t* held;         // [rows][ldz]: e, or dz made of it
  uint16_t* xs;           // [rows][ldxc]: f x; NULL: not wanted (never where dz is made)
  float* factor;          // [rows]: f; where dz is made, 0 of an ignored row and else 1
  int64_t ldz;
  int32_t vec;            // x and w are read in vectors
  int32_t alone;          // rows that want another reference are made anew by their block (kOnce)
  // Rows that are not ignored, one after the other (NULL: all rows as they are):
  int32_t* place;         // [rows]: the piece's row that the k-th is
  int32_t* slot;          // [rows]: and the k that a row is, -1: ignored
  int64_t fill;           // rows that are 0 behind them at least, from the first on
  uint16_t* dxc;          // [rows][lddxc]: their dx
  int64_t lddxc;
  uint16_t* dx;           // the piece's
  int64_t lddx;
  int32_t dx_vec;
  int32_t direct;         // dx is written where it belongs if no row is ignored
};

// The rows of a piece that the kernels look at: those there are, and those that are 0.
__device__ __forceinline__ int64_t rows_of(const LossArgs& a) {
  return a.place != nullptr ? __ldcg(&a.words->rows) : a.rows;
}
__device__ __forceinline__ int64_t filled_rows(const LossArgs& a, int64_t n) {
  if (a.place == nullptr) return a.rows;
  int64_t m = (n + 127) / 128 * 128;
  m = m > a.fill ? m : a.fill;
  return m < a.rows ? m : a.rows;
}

__device__ __forceinline__ int64_t target_of(const LossArgs& a, int64_t i) {
  return a.ids_i32 ? static_cast<const int32_t*>(a.targets)[i]
                   : static_cast<const int64_t*>(a.targets)[i];
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int k = 16; k > 0; k /= 2) x += __shfl_xor_sync(0xffffffffu, x, k);
  return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int k = 16; k > 0; k /= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
  return x;
}

// Where the rows that are not ignored go: one after the other, so that the products have no
// others to do.  One block: a warp looks through a run of rows, once to count and once to
// write (8,192 rows: 4 us).
constexpr int kPlaceWarps = 32;
__global__ void __launch_bounds__(32 * kPlaceWarps) loss_places_kernel(const __grid_constant__ LossArgs a) {
  __shared__ int32_t found[kPlaceWarps];
  wait_for_predecessor();
  launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t each = (a.rows + 32 * kPlaceWarps - 1) / (32 * kPlaceWarps) * 32;
  const int64_t from = warp * each < a.rows ? warp * each : a.rows, to = from + each < a.rows ? from + each : a.rows;
  constexpr int U = 8;
  const auto look = [&](auto f) {
    for (int64_t i0 = from; i0 < to; i0 += 32 * U) {
      int64_t t[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + 32 * u + lane;
        t[u] = target_of(a, a.first + (i < to ? i : to - 1));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + 32 * u + lane;
        f(i, i < to && t[u] != a.ignore);
      }
    }
  };
  int n = 0;
  look([&](int64_t, bool has) { n += __popc(__ballot_sync(0xffffffffu, has)); });
  if (lane == 0) found[warp] = n;
  __syncthreads();
  int at = 0, all = 0;
  for (int w = 0; w < kPlaceWarps; ++w) {
    if (w < warp) at += found[w];
    all += found[w];
  }
  look([&](int64_t i, bool has) {
    const uint32_t those = __ballot_sync(0xffffffffu, has);
    const int k = at + __popc(those & ((1u << lane) - 1u));
    if (i < to) {
      a.slot[i] = has ? k : -1;
      if (has) a.place[k] = static_cast<int32_t>(i);
      else a.losses[a.first + i] = 0.0f;
    }
    at += __popc(those);
  });
  if (threadIdx.x == 0) *a.words = Words{0, 0, all, 0.0f};
}

// A lane's part of the product of two rows of bf16; f(j, v) is given x's vectors or elements.
template <bool VEC, typename F>
__device__ __forceinline__ float dot_part(const uint16_t* x, const uint16_t* w, int64_t width, int lane, F f) {
  float sum = 0.0f;
  if constexpr (VEC) {
    int64_t j = 8 * lane;
    const auto add = [&](uint4 v, uint4 u) {
      float p[8], q[8];
      bf16x8(v, p);
      bf16x8(u, q);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum = fmaf(p[c], q[c], sum);
    };
    constexpr int U = 4;  // of each row's loads under way
    for (; j + 256 * (U - 1) + 8 <= width; j += 256 * U) {
      uint4 v[U], u[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        v[k] = __ldg(reinterpret_cast<const uint4*>(x + j + 256 * k));
        u[k] = __ldg(reinterpret_cast<const uint4*>(w + j + 256 * k));
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        add(v[k], u[k]);
        f(j + 256 * k, v[k]);
      }
    }
    for (; j + 8 <= width; j += 256) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + j));
      add(v, __ldg(reinterpret_cast<const uint4*>(w + j)));
      f(j, v);
    }
    for (; j < width; ++j) {  // (one lane's: what is left of a vector)
      sum = fmaf(bf16_at(x + j), bf16_at(w + j), sum);
      f(j, x[j]);
    }
  } else {
    for (int64_t j = lane; j < width; j += 32) {
      sum = fmaf(bf16_at(x + j), bf16_at(w + j), sum);
      f(j, x[j]);
    }
  }
  return sum;
}

struct Nothing {
  __device__ __forceinline__ void operator()(int64_t, uint4) const {}
  __device__ __forceinline__ void operator()(int64_t, uint16_t) const {}
};

// A warp a row: the target's logit, and x laid out for TMA, an ignored row's as zeros
// (its x may hold anything, and 0 times an infinity would reach dw).
template <bool VEC>
__global__ void __launch_bounds__(256) loss_rows_kernel(const __grid_constant__ LossArgs a) {
  wait_for_predecessor();
  launch_dependents();
  if (a.place == nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.words = Words{0, 0, 0, 0.0f};
  const int lane = threadIdx.x % 32;
  const int64_t n = rows_of(a), filled = filled_rows(a, n);
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; k < filled;
       k += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t i = a.first + (a.place == nullptr ? k : k < n ? __ldcg(a.place + k) : 0);
    const int64_t t = target_of(a, i);
    const bool ignored = k >= n || t == a.ignore, column = !ignored && t >= 0 && t < a.vocab;
    uint16_t* to = a.xc + k * a.ldxc;
    float sum = 0.0f;
    if (ignored) {  // (the pitch has room for whole vectors)
      for (int64_t j = 8 * lane; j < a.width; j += 256) *reinterpret_cast<uint4*>(to + j) = make_uint4(0, 0, 0, 0);
    } else {
      struct Put {
        uint16_t* to;
        __device__ __forceinline__ void operator()(int64_t j, uint4 v) const { *reinterpret_cast<uint4*>(to + j) = v; }
        __device__ __forceinline__ void operator()(int64_t j, uint16_t v) const { to[j] = v; }
      };
      sum = dot_part<VEC>(a.x + i * a.ldx, a.w + (column ? t : 0) * a.ldw, a.width, lane, Put{to});
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      const float zt = column || ignored ? sum : NAN;
      a.zt[k] = zt;
      a.ref[k] = isfinite(zt) ? zt : 0.0f;
      a.column[k] = column ? static_cast<int32_t>(t) : ignored ? -1 : -2;
    }
  }
}

constexpr int kFinishThreads = 256, kFinishWarps = kFinishThreads / 32;

// Whether this is the last of the grid's blocks; all that the others wrote can be read then.
__device__ __forceinline__ bool last_block(Words* words, int32_t* shared) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *shared = atomicAdd(&words->ticket, 1) == static_cast<int32_t>(gridDim.x) - 1;
  __syncthreads();
  __threadfence();
  return *shared != 0;
}

// The rows that count, and with `sums` their losses' sum, of all pieces: in 64 bits, in an order
// that follows from the sizes.  A whole block.
__device__ __forceinline__ void total_losses(const LossArgs& a, bool sums) {
  __shared__ double sum_part[kFinishWarps];
  __shared__ int32_t count_part[kFinishWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  double total = 0.0;
  int32_t valid = 0;
  // Where the rows that count are counted, and c is alike for all: the losses alone, an ignored
  // row's being 0.
  const bool counted = a.place != nullptr && a.rows == a.all_rows && a.scale == nullptr;
  if (counted) {
    constexpr int U = 16;
    valid = threadIdx.x == 0 ? __ldcg(&a.words->rows) : 0;
    for (int64_t i0 = threadIdx.x; sums && i0 < a.all_rows; i0 += U * kFinishThreads) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = i0 + u * kFinishThreads < a.all_rows ? __ldcg(a.losses + i0 + u * kFinishThreads) : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) total += static_cast<double>(x[u]);
    }
  }
  constexpr int U = 8;
  for (int64_t i0 = threadIdx.x; !counted && i0 < a.all_rows; i0 += U * kFinishThreads) {
    float x[U], c[U];
    int64_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kFinishThreads < a.all_rows ? i0 + u * kFinishThreads : i0;
      t[u] = target_of(a, i);
      x[u] = sums ? __ldcg(a.losses + i) : 0.0f;
      c[u] = a.scale != nullptr ? __ldg(a.scale + i) : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kFinishThreads < a.all_rows && t[u] != a.ignore) {
        ++valid;
        total += static_cast<double>(c[u]) * static_cast<double>(x[u]);
      }
  }
#pragma unroll
  for (int k = 16; k > 0; k /= 2) total += __shfl_xor_sync(0xffffffffu, total, k);
  valid = __reduce_add_sync(0xffffffffu, valid);
  if (lane == 0) {
    sum_part[warp] = total;
    count_part[warp] = valid;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  total = 0.0;
  valid = 0;
  for (int k = 0; k < kFinishWarps; ++k) {
    total += sum_part[k];
    valid += count_part[k];
  }
  a.words->share = valid > 0 ? 1.0f / static_cast<float>(valid) : 0.0f;
  if (a.scale == nullptr) total = valid > 0 ? total / valid : 0.0;
  if (sums) *a.total = static_cast<float>(total);
}

// The loss alone, a warp a row: of parts less their own largest logit.
template <bool VEC>
__global__ void __launch_bounds__(kFinishThreads) loss_alone_kernel(const __grid_constant__ LossArgs a) {
  __shared__ int32_t last;
  wait_for_predecessor();
  launch_dependents();
  const int lane = threadIdx.x % 32;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kFinishWarps + threadIdx.x / 32; i < a.rows;
       i += static_cast<int64_t>(gridDim.x) * kFinishWarps) {
    const int64_t t = target_of(a, a.first + i);
    const bool column = t >= 0 && t < a.vocab;
    if (t == a.ignore || !column) {
      if (lane == 0) a.losses[a.first + i] = t == a.ignore ? 0.0f : NAN;
      continue;
    }
    const float zt = warp_sum(dot_part<VEC>(a.x + (a.first + i) * a.ldx, a.w + t * a.ldw, a.width, lane, Nothing{}));
    const float2* parts = a.sums + i * a.parts;
    // a lane's parts, less the largest logit of them so far
    float top = -INFINITY, sum = 0.0f;
    constexpr int U = 4;
    for (int k0 = lane; k0 < a.parts; k0 += 32 * U) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = k0 + 32 * u < a.parts ? __ldcg(parts + k0 + 32 * u) : make_float2(0.0f, -INFINITY);
      float now = top;
#pragma unroll
      for (int u = 0; u < U; ++u) now = fmaxf(now, v[u].y);
      if (sum != 0.0f) sum *= expf(top - now);
      top = now;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v[u].x != 0.0f) sum += v[u].x * expf(v[u].y - now);
    }
    float most = fmaxf(top, zt);
#pragma unroll
    for (int k = 16; k > 0; k /= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
    // less the target's logit, where that leaves fp32's range alone: 2^31 columns of e^44 come to
    // 3e28 (of e^80, 1e5 columns already pass 3.4e38)
    const bool own = most - zt < 44.0f;
    const float ref = own ? zt : most;
    if (sum != 0.0f) sum *= expf(top - ref);
    sum = warp_sum(sum);
    if (lane == 0) a.losses[a.first + i] = own ? log1pf(sum) : (ref - zt) + logf(sum + expf(zt - ref));
  }
  if (a.total != nullptr && last_block(a.words, &last)) total_losses(a, true);
}

// Row i's exponentials less `ref`, as the product's epilogue makes them, by WARPS warps; this warp's
// part of their sum.  Four columns at a time.
template <bool VEC, int WARPS>
__device__ __noinline__ float row_again(const LossArgs& a, int64_t i, int32_t t, float ref) {
  const int warp = threadIdx.x / 32 % WARPS, lane = threadIdx.x % 32;
  const uint16_t* x = a.xc + i * a.ldxc;
  constexpr int U = 4;
  float sum = 0.0f;
  for (int64_t j = U * warp; j < a.vocab; j += U * WARPS) {
    const uint16_t* w[U];
    float z[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = a.w + (j + u < a.vocab ? j + u : j) * a.ldw;
    if constexpr (VEC) {
      int64_t k = 8 * lane;
      for (; k + 8 <= a.width; k += 256) {
        float p[8];
        bf16x8(__ldg(reinterpret_cast<const uint4*>(x + k)), p);
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = __ldg(reinterpret_cast<const uint4*>(w[u] + k));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float q[8];
          bf16x8(v[u], q);
#pragma unroll
          for (int c = 0; c < 8; ++c) z[u] = fmaf(p[c], q[c], z[u]);
        }
      }
      for (; k < a.width; ++k)  // (one lane's: what is left of a vector)
#pragma unroll
        for (int u = 0; u < U; ++u) z[u] = fmaf(bf16_at(x + k), bf16_at(w[u] + k), z[u]);
    } else {
      for (int64_t k = lane; k < a.width; k += 32)
#pragma unroll
        for (int u = 0; u < U; ++u) z[u] = fmaf(bf16_at(x + k), bf16_at(w[u] + k), z[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      z[u] = warp_sum(z[u]);
      if (j + u >= a.vocab) continue;
      const float d = j + u == t ? -INFINITY : z[u] - ref;
      sum += expf(d);
      if (lane == 0) a.held[i * a.ldz + j + u] = to_bf16(expf(d));
    }
  }
  return sum;
}

// A row's sums in the order of its parts, its loss, e of the target, and f: with DZ f times e in
// place, a block a row, without it f times x, a warp a row.  The last block adds up the losses.  With
// c alike for all rows (the mean) c is left to the products' sums, and dz is p less the target's 1,
// whose rounding is nothing where p is small.
// Without DZ bound by HBM: the sums, x twice (8192 x 2048 -> 50257: 100 MB).
// Where the whole product is small, a row that wants another reference is made anew here, by
// dot products, which saves the two launches that else do it (37 x 256 -> 515: 5 us of 37); such
// a row takes its block some 30 us at most.
constexpr int64_t kFewProducts = int64_t{1} << 28, kFewWeights = int64_t{1} << 21;
constexpr int64_t kFewValues = int64_t{1} << 25;
// (Warps instead of blocks: 8192 x 256 -> 100 77 -> 47 us, 4096 x 768 -> 4000 103 -> 90, 700 x 512 -> 4000 50.5
// and 50.8.)
constexpr int64_t kWarpRows = 600, kWarpVocab = 4096, kFewColumns = 64;

enum Time { kFirst, kAgain, kOnce };

template <Time TIME, bool DZ, int WARPS>
__global__ void __launch_bounds__(kFinishThreads) loss_ends_kernel(const __grid_constant__ LossArgs a) {
  static_assert(TIME != kOnce || DZ);
  __shared__ float2 part[kFinishWarps];
  __shared__ int32_t last;
  wait_for_predecessor();
  launch_dependents();
  if (TIME == kAgain && __ldcg(&a.words->again) == 0) return;
  constexpr int kThreads = 32 * WARPS;  // of a row
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, thread = threadIdx.x % kThreads;
  const int64_t n = rows_of(a), filled = filled_rows(a, n);
  if constexpr (!DZ) {  // e of the rows behind the last: zeros, by the whole grid (43 rows of 50257 columns, a warp a row: 5 us)
    const int64_t vectors = (a.vocab + 7) / 8;
    for (int64_t i = n; i < filled; ++i)
      for (int64_t j = blockIdx.x * kFinishThreads + threadIdx.x; j < vectors; j += gridDim.x * kFinishThreads)
        reinterpret_cast<uint4*>(a.held + i * a.ldz)[j] = make_uint4(0, 0, 0, 0);
  }
  constexpr int kRows = kFinishWarps / WARPS;  // of a block at one time
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kThreads; i < filled;
       i += static_cast<int64_t>(gridDim.x) * kRows) {
    const int32_t t = __ldcg(a.column + i);
    const int64_t from = a.first + (a.place == nullptr ? i : i < n ? __ldcg(a.place + i) : 0);  // the caller's row
    const float zt = __ldcg(a.zt + i);
    float ref = __ldcg(a.ref + i), sum = 0.0f, top = -INFINITY;
    if (a.place != nullptr ? i < n : t != -1) {  // (the same; with i nothing waits for t)
      constexpr int U = 8;
      for (int k0 = thread; k0 < a.parts; k0 += U * kThreads) {
        float2 s[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          s[u] = k0 + u * kThreads < a.parts ? __ldcg(a.sums + i * a.parts + k0 + u * kThreads)
                                             : make_float2(0.0f, -INFINITY);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          sum += s[u].x;
          top = fmaxf(top, s[u].y);
        }
      }
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int k = 16; k > 0; k /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    const auto of_block = [&] {  // (the warps' sums in their order)
      __syncthreads();  // the row before is done with part[]; what row_again wrote is there
      if (lane == 0) part[warp] = make_float2(sum, top);
      __syncthreads();
      sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kFinishWarps; ++k) {
        sum += part[k].x;
        top = fmaxf(top, part[k].y);
      }
    };
    if constexpr (WARPS > 1) of_block();
    if (TIME != kAgain && t >= 0 && sum > kOneMore && isfinite(top)) {
      if constexpr (TIME == kOnce) {
        ref = top;
        sum = a.vec ? row_again<true, WARPS>(a, i, t, ref) : row_again<false, WARPS>(a, i, t, ref);
        if constexpr (WARPS > 1) of_block();
        else __syncwarp();  // (the row is written)
      } else if (lane == 0) {
        a.ref[i] = top;
        a.words->again = 1;
      }
    }
    const bool own = zt == ref;
    const float et = own ? 1.0f : expf(zt - ref);
    const float whole = sum + et;
    float loss = own ? log1pf(sum) : (ref - zt) + logf(whole);
    // a NaN is no column's, or of the inputs'; an infinite logit leaves no gradient
    float f = (a.scale != nullptr ? __ldg(a.scale + from) : 1.0f) / whole;
    if (!isfinite(whole)) f = NAN;
    if (t == -1) loss = f = 0.0f;
    if (t == -2) loss = f = NAN;
    if (thread == 0 && i < n) a.losses[from] = loss;
    if constexpr (DZ) {
      // where ignored rows are not left out: 0 times an infinite weight would reach dx
      if (thread == 0) a.factor[i] = t == -1 ? 0.0f : 1.0f;
      // (the pitch has room for whole vectors; an ignored row's e are not read)
      uint4* e = reinterpret_cast<uint4*>(a.held + i * a.ldz);
      constexpr int U = 4;
      const uint32_t vectors = static_cast<uint32_t>((a.vocab + 7) / 8);
      // Where few columns share a row, e's roundings do not average out.  One of at least half of their
      // sum takes what makes the sum, as rounded, S' again: that is at most another rounding of its own,
      // as the others weigh no more than it; with a factor for all, small ones could be off by two
      // more.  (100 rows, 2 columns: dx and dw 1.4 times as far from 64 bits as their own rounding puts
      // them, without this 1.55; 12 x 2048 -> 2 1.25, at worst 1.8, and 1.5, 2.8.)
      if (a.vocab <= kFewColumns) {
        if (thread >= 32) continue;  // (its vectors are its first warp's lanes')
        const uint32_t j = thread, at = static_cast<uint32_t>(t) - 8 * j;
        float x[8] = {}, held = 0.0f, most = 0.0f;
        if (t != -1 && j < vectors) bf16x8(__ldcg(e + j), x);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (8 * j + c >= a.vocab) x[c] = 0.0f;  // (nothing was written there)
          held += x[c];
          most = fmaxf(most, x[c]);
        }
        held = warp_sum(held);
        const float top_e = warp_max(most);
        const uint32_t those = __ballot_sync(0xffffffffu, most == top_e);
        if (top_e > 0.0f && 2.0f * top_e >= held && __ffs(those) - 1 == lane) {
          bool done = false;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (!done && x[c] == top_e) {
              x[c] += sum - held;
              done = true;
            }
        }
        if (j < vectors) {
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] = t == -1 ? 0.0f : at == c ? -(f * sum) : f * x[c];
          e[j] = to_bf16x8(x);
        }
        continue;
      }
      for (uint32_t j0 = thread; j0 < vectors; j0 += U * kThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (t != -1 && j0 + u * kThreads < vectors) v[u] = __ldcg(e + j0 + u * kThreads);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t j = j0 + u * kThreads, at = static_cast<uint32_t>(t) - 8 * j;
          if (j >= vectors) break;
          float x[8] = {};
          if (t != -1) bf16x8(v[u], x);
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] = t == -1 ? 0.0f : at == c ? -(f * sum) : f * x[c];
          e[j] = to_bf16x8(x);
        }
      }
    } else {
      // f takes what e_t's rounding loses: f e_t is then exact, and the others, which weigh less
      // together, are off by as much as one more rounding of theirs
      const float rounded = __uint_as_float(static_cast<uint32_t>(to_bf16(sum)) << 16);
      if (t >= 0 && rounded > 0.0f) f *= sum / rounded;
      if (thread == 0) {
        a.factor[i] = f;
        if (t >= 0) a.held[i * a.ldz + t] = to_bf16(-sum);
      }
      if (a.xs == nullptr) continue;
      const uint16_t* x = a.xc + i * a.ldxc;
      uint16_t* to = a.xs + i * a.ldxc;
#pragma unroll 4
      for (int64_t j = 8 * thread; j < a.width; j += 8 * kThreads) {
        float p[8];
        bf16x8(__ldcg(reinterpret_cast<const uint4*>(x + j)), p);
#pragma unroll
        for (int c = 0; c < 8; ++c) p[c] *= f;
        *reinterpret_cast<uint4*>(to + j) = to_bf16x8(p);
      }
    }
  }
  if (!last_block(a.words, &last)) return;
  if (TIME == kFirst && threadIdx.x == 0) a.words->ticket = 0;
  // (the losses are complete after the second time, where there is one)
  total_losses(a, a.total != nullptr && (TIME != kFirst || __ldcg(&a.words->again) == 0));
}

// dx of every row of the piece from those that are not ignored; the others' is 0.  A warp a row.
__global__ void __launch_bounds__(256) loss_spread_kernel(const __grid_constant__ LossArgs a) {
  wait_for_predecessor();
  launch_dependents();
  if (a.direct && __ldcg(&a.words->rows) == a.rows) return;
  const int lane = threadIdx.x % 32;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; i < a.rows;
       i += static_cast<int64_t>(gridDim.x) * 8) {
    const int32_t k = __ldcg(a.slot + i);
    const uint16_t* from = a.dxc + (k < 0 ? 0 : k) * a.lddxc;
    uint16_t* to = a.dx + i * a.lddx;
    if (a.dx_vec) {
#pragma unroll 4
      for (int64_t j = 8 * lane; j + 8 <= a.width; j += 256)
        *reinterpret_cast<uint4*>(to + j) =
            k < 0 ? make_uint4(0, 0, 0, 0) : __ldcs(reinterpret_cast<const uint4*>(from + j));
      for (int64_t j = a.width / 8 * 8 + lane; j < a.width; j += 32) to[j] = k < 0 ? 0 : from[j];
    } else {
#pragma unroll 4
      for (int64_t j = lane; j < a.width; j += 32) to[j] = k < 0 ? 0 : from[j];
    }
  }
}

// dw (bf16) from the pieces' fp32 sums.
__global__ void __launch_bounds__(256) loss_round_kernel(const float* from, int64_t ldf, uint16_t* to,
                                                         int64_t ldt, int64_t rows, int64_t cols,
                                                         int32_t accumulate) {
  wait_for_predecessor();
  launch_dependents();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t j = threadIdx.x; j < cols; j += 256) {
      const float x = __ldcs(from + r * ldf + j);
      uint16_t* o = to + r * ldt + j;
      *o = to_bf16(accumulate ? bf16_at(o) + x : x);
    }
}

// Rows of a piece.
int64_t piece_rows(const zero_cross_entropy_t& s, bool grads) {
  const int64_t row = grads ? 2 * laid_out_pitch(s.vocab) : 16 * ((s.vocab + 127) / 128);
  int64_t n = kMostHeld / row / 256 * 256;
  if (n < 256) n = 256;
  return s.rows < n ? s.rows : n;
}

// Where a call's arrays lie in its workspace.
struct Layout {
  int64_t piece, parts;  // rows of a piece, and parts of the vocabulary at most
  int64_t w, x, xs, zt, held, sums, losses, acc, dxc, linear, bytes;
};

zero_linear_t linear_of(const zero_cross_entropy_t& s, int64_t rows) {
  zero_linear_t l{};
  l.rows = rows;
  l.in = s.width;
  l.out = s.vocab;
  l.ldx = laid_out_pitch(s.width);
  l.ldy = laid_out_pitch(s.vocab);
  l.lddx = s.lddx;
  l.lddw = s.lddw;
  return l;
}

struct LayoutKey {
  int64_t rows, width, vocab;
  int32_t flags;
  bool operator==(const LayoutKey& o) const {
    return rows == o.rows && width == o.width && vocab == o.vocab && flags == o.flags;
  }
};

Layout make_layout(const zero_cross_entropy_t& s, int32_t flags) {
  const bool grads = (flags & ZERO_LINEAR_BACKWARD) != 0;
  Layout l{};
  l.piece = piece_rows(s, grads);
  const int64_t rest = l.piece > 0 ? s.rows % l.piece : 0;
  if (s.rows > 0) {
    l.parts = exponent_parts(l.piece, s.vocab, s.width);
    const int64_t more = rest > 0 ? exponent_parts(rest, s.vocab, s.width) : 0;
    l.parts = more > l.parts ? more : l.parts;
  }
  int64_t at = 256;  // Words
  const auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += round_up(bytes, 256);
    return p;
  };
  l.w = take((flags & ZERO_LINEAR_ALIGNED) ? 0 : 2 * s.vocab * laid_out_pitch(s.width));
  // (the loss alone reads x in place, if it lies so; what it lies like is not known here)
  l.x = take(2 * l.piece * laid_out_pitch(s.width));
  l.xs = take(grads && l.piece * s.vocab > kFewValues ? 2 * l.piece * laid_out_pitch(s.width) : 0);
  l.zt = take(24 * l.piece);  // zt, ref, column, place, slot, factor
  l.held = take(grads ? 2 * l.piece * laid_out_pitch(s.vocab) : 0);
  l.sums = take(8 * l.piece * l.parts);
  l.losses = take(4 * s.rows);
  const bool sums32 = grads && s.rows > l.piece && (flags & ZERO_GRAD_F32) == 0;
  l.acc = take(sums32 ? 4 * s.vocab * round_up(s.width, 4) : 0);
  l.dxc = take(grads ? 2 * l.piece * laid_out_pitch(s.width) : 0);
  l.linear = at;
  if (grads && s.rows > 0) {
    constexpr int32_t kind = ZERO_LINEAR_BACKWARD | ZERO_LINEAR_ALIGNED | ZERO_LINEAR_PLAIN;
    int64_t need = linear_workspace(linear_of(s, l.piece), kind);
    const int64_t more = rest > 0 ? linear_workspace(linear_of(s, rest), kind) : 0;
    at += round_up(need > more ? need : more, 256);
  }
  l.bytes = at;
  return l;
}

Layout layout_of(const zero_cross_entropy_t& s, int32_t flags) {
  static thread_local Memo<LayoutKey, Layout> memo;
  return memo.get({s.rows, s.width, s.vocab, flags}, [&] { return make_layout(s, flags); });
}

}  // namespace

int64_t cross_entropy_workspace(const zero_cross_entropy_t& s, int32_t flags) {
  return layout_of(s, flags).bytes;
}

cudaError_t launch_cross_entropy(const CrossEntropyLaunch& L) {
  (void)cudaGetLastError();
  const zero_cross_entropy_t& s = L.s;
  const bool grads = L.dx != nullptr || L.dw != nullptr;
  const bool in_place = tileable_matrix(L.w, s.vocab, s.width, s.ldw);
  const Layout l = layout_of(s, (grads ? ZERO_LINEAR_BACKWARD : 0) | (in_place ? ZERO_LINEAR_ALIGNED : 0) |
                                    (L.grad_f32 ? ZERO_GRAD_F32 : 0));
  char* base = static_cast<char*>(L.workspace);
  if (s.rows == 0) {
    cudaError_t e = L.total != nullptr ? cudaMemsetAsync(L.total, 0, 4, L.stream) : cudaSuccess;
    if (e != cudaSuccess || L.dw == nullptr || L.accumulate) return e;
    const int64_t size = L.grad_f32 ? 4 : 2;
    return cudaMemset2DAsync(L.dw, s.lddw * size, 0, s.width * size, s.vocab, L.stream);
  }
  Chain chain{L.stream};
  LossArgs a{};
  a.x = L.x;
  a.w = L.w;
  a.ldx = s.ldx;
  a.ldw = s.ldw;
  a.targets = L.targets;
  a.ids_i32 = L.ids_i32;
  a.ignore = L.ignore;
  a.all_rows = s.rows;
  a.width = s.width;
  a.vocab = s.vocab;
  a.words = reinterpret_cast<Words*>(base);
  a.zt = reinterpret_cast<float*>(base + l.zt);
  a.ref = a.zt + l.piece;
  a.column = reinterpret_cast<int32_t*>(a.ref + l.piece);
  int32_t* const place = a.column + l.piece;
  a.slot = place + l.piece;
  a.factor = reinterpret_cast<float*>(a.slot + l.piece);
  a.dxc = reinterpret_cast<uint16_t*>(base + l.dxc);
  a.lddxc = laid_out_pitch(s.width);
  a.lddx = s.lddx;
  a.dx_vec = aligned(L.dx, 16) && s.lddx % 8 == 0;
  a.xc = reinterpret_cast<uint16_t*>(base + l.x);
  a.ldxc = laid_out_pitch(s.width);
  a.sums = reinterpret_cast<const float2*>(base + l.sums);
  a.scale = L.scale;
  a.losses = L.losses != nullptr ? L.losses : reinterpret_cast<float*>(base + l.losses);
  a.held = reinterpret_cast<uint16_t*>(base + l.held);
  a.ldz = laid_out_pitch(s.vocab);
  a.vec = aligned(L.x, 16) && aligned(L.w, 16) && (s.rows == 1 || s.ldx % 8 == 0) &&
          (s.vocab == 1 || s.ldw % 8 == 0);
  const uint16_t* w = L.w;
  int64_t ldw = s.ldw;
  cudaError_t e = cudaSuccess;
  if (!in_place) {
    uint16_t* copy = reinterpret_cast<uint16_t*>(base + l.w);
    e = launch_lay_out(w, s.vocab, s.width, ldw, copy, L.stream);
    w = copy;
    ldw = laid_out_pitch(s.width);
  }
  const bool joined = L.dw != nullptr && s.rows > l.piece && !L.grad_f32;  // sums of pieces in fp32
  float* acc = reinterpret_cast<float*>(base + l.acc);
  const auto blocks_of = [](int64_t n, int64_t most) {
    return dim3(static_cast<unsigned>(n < most ? n : most));
  };
  for (int64_t first = 0; e == cudaSuccess && first < s.rows; first += l.piece) {
    a.first = first;
    a.rows = s.rows - first < l.piece ? s.rows - first : l.piece;
    const bool last = first + a.rows == s.rows;
    a.alone = a.rows * s.vocab <= kFewProducts / s.width && s.vocab <= kFewWeights / s.width;
    a.parts = static_cast<int32_t>(exponent_parts(a.rows, s.vocab, s.width));
    a.total = last ? L.total : nullptr;
    const bool make_dz = a.alone || a.rows * s.vocab <= kFewValues;
    a.xs = L.dw != nullptr && !make_dz ? reinterpret_cast<uint16_t*>(base + l.xs) : nullptr;
    ExponentLaunch x{};
    x.rows = a.rows;
    x.width = s.width;
    x.vocab = s.vocab;
    x.w = w;
    x.ldw = ldw;
    x.stream = L.stream;
    x.withhold = L.withhold;
    x.of.sums = const_cast<float2*>(a.sums);
    x.of.sum_pitch = a.parts;
    if (!grads) {
      x.x = L.x + first * s.ldx;
      x.ldx = s.ldx;
      if (!tileable_matrix(x.x, a.rows, s.width, s.ldx)) {
        e = launch_lay_out(x.x, a.rows, s.width, s.ldx, a.xc, L.stream);
        x.x = a.xc;
        x.ldx = a.ldxc;
      }
      x.of.targets = static_cast<const char*>(L.targets) + first * (L.ids_i32 ? 4 : 8);
      x.of.ids_i32 = L.ids_i32;
      x.of.ignore = L.ignore;
      x.of.ticket = &a.words->ticket;
      if (e == cudaSuccess) e = launch_exponents(x);
      if (e == cudaSuccess)
        e = chain.launch(a.vec ? loss_alone_kernel<true> : loss_alone_kernel<false>, blocks_of((a.rows + kFinishWarps - 1) / kFinishWarps, 8 * kSms),
                         kFinishThreads, 0, 1, a);
      continue;
    }
    a.place = a.alone ? nullptr : place;
    zero_linear_t b_shape = linear_of(s, a.rows);
    a.fill = L.dw != nullptr ? least_rows(b_shape, L.dx != nullptr) : 0;
    a.dx = L.dx != nullptr ? L.dx + first * s.lddx : nullptr;
    if (!a.alone) e = chain.launch(loss_places_kernel, dim3(1), 32 * kPlaceWarps, 0, 1, a);
    if (e == cudaSuccess)
      e = chain.launch(a.vec ? loss_rows_kernel<true> : loss_rows_kernel<false>,
                     blocks_of((a.rows + 7) / 8, 16 * kSms), 256, 0, 1, a);
    x.x = a.xc;
    x.ldx = a.ldxc;
    x.of.ref = a.ref;
    x.of.target = a.column;
    x.out = a.held;
    x.ldo = a.ldz;
    x.rows_now = a.alone ? nullptr : &a.words->rows;
    if (e == cudaSuccess) e = launch_exponents(x);
    const bool warps = !make_dz || (a.rows > kWarpRows && s.vocab <= kWarpVocab);  // a warp a row
    const dim3 grid = blocks_of(warps ? (a.rows + kFinishWarps - 1) / kFinishWarps : a.rows, 8 * kSms);
    const auto end = [&](auto first_time) {
      constexpr Time TIME = decltype(first_time)::value ? kFirst : kAgain;
      return chain.launch(!make_dz ? loss_ends_kernel<TIME, false, 1>
                          : warps  ? loss_ends_kernel<TIME, true, 1>
                                   : loss_ends_kernel<TIME, true, kFinishWarps>,
                          grid, kFinishThreads, 0, 1, a);
    };
    if (e == cudaSuccess && a.alone)
      e = chain.launch(warps ? loss_ends_kernel<kOnce, true, 1> : loss_ends_kernel<kOnce, true, kFinishWarps>, grid,
                       kFinishThreads, 0, 1, a);
    if (!a.alone) {
      if (e == cudaSuccess) e = end(std::true_type{});
      x.of.only_if = &a.words->again;
      if (e == cudaSuccess) e = launch_exponents(x);
      if (e == cudaSuccess) e = end(std::false_type{});
    }
    if (e != cudaSuccess) return e;
    LinearBackwardLaunch b{};
    b.s = b_shape;
    b.s.ldw = ldw;
    b.dy = a.held;
    b.x = make_dz ? a.xc : a.xs;
    b.w = w;
    b.dx = a.dx;
    if (a.dx != nullptr && !a.alone) {
      a.direct = a.dx_vec && a.rows > 1 && whole_in_place(b.s, L.dw != nullptr);
      if (a.direct) {
        b.dx_all = a.dx;
        b.ld_all = s.lddx;
      }
      b.dx = a.dxc;
      b.s.lddx = a.lddxc;
    }
    b.rows_now = x.rows_now;
    b.dw = joined ? acc : L.dw;
    if (joined) b.s.lddw = round_up(s.width, 4);
    b.grad_f32 = L.grad_f32 || joined;
    b.accumulate = first > 0 || (L.accumulate && !joined);
    b.row_scale = make_dz && !a.alone ? nullptr : a.factor;
    b.scale = L.scale == nullptr ? &a.words->share : nullptr;
    b.workspace = base + l.linear;
    b.stream = L.stream;
    b.withhold = L.withhold;
    e = launch_linear_backward(b);
    if (e == cudaSuccess && a.dx != nullptr && !a.alone)
      e = chain.launch(loss_spread_kernel, blocks_of((a.rows + 7) / 8, 16 * kSms), 256, 0, 1, a);
  }
  if (e == cudaSuccess && joined)
    e = chain.launch(loss_round_kernel, blocks_of(s.vocab, 16 * kSms), 256, 0, 1, acc,
                     round_up(s.width, 4), static_cast<uint16_t*>(L.dw), s.lddw, s.vocab, s.width,
                     L.accumulate);
  return e;
}

}  // namespace zeroadam
