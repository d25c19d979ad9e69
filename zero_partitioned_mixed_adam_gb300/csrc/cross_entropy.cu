// cross_entropy.cu -- softmax cross entropy of a linear map onto a vocabulary, and
// its gradients, on sm_103a.
//
// With z = x W^T, a row's loss is log(sum over j of exp(z_j)) - z_t.  z is never kept.
// A row's exponentials are taken less a reference r that is there before the product:
// the target's logit z_t itself, one dot product a row.  Then, S' the sum over j != t,
//   loss = log(1 + S'),   p_j = exp(z_j - z_t) / (1 + S'),   1 - p_t = S' / (1 + S'),
// where nothing is lost to cancellation however sure the model is.  The gradient
// dz_j = c (p_j - [j = t]) wants the row's whole sum first, so the product's epilogue
// writes z_j - z_t in 16 bits, and one pass over them makes dz of them in place once the
// sums are there: three products for the loss and both gradients, where computing z
// again would be a fourth (8192 x 2048 -> 50257: 0.9 ms; the pass 0.25).
// A row whose S' passes 2^44 (the target 30 below the largest logit) leaves that range:
// its reference becomes the largest logit, which the first product found, and product and
// pass run once more; the launches that do so end at once where no row needs them.
//
// Kernels of one piece of rows:
//   rows      z_t, the reference, the target as a column, x where TMA can read it
//   product   (linear.cu) exponentials
//   finish    losses, dz;  product and finish again, where some row needs it
//   products  (linear.cu) dx = dz W, dw = dz^T x
#include "chain.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

constexpr int64_t kMostHeld = int64_t{1} << 30;  // bytes of 16-bit values of one piece
constexpr float kOneMore = 17592186044416.0f;    // 2^44: a sum that asks for another reference

// Words of the workspace that a call's kernels share.
struct Words {
  int32_t again;   // some row of this piece wants another reference
  int32_t ticket;  // blocks of the last kernel that are done
  int32_t valid;   // rows that are not ignored, of all pieces
  float share;     // 1 / valid: c of the mean (0 where there is none)
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
  float* total;           // NULL: not wanted, or not the last piece
  uint16_t* held;         // [rows][ldz]: 16 bits, then dz; NULL: no gradients
  int64_t ldz;
  int32_t vec;            // x and w are read in vectors
};

__device__ __forceinline__ int64_t target_of(const LossArgs& a, int64_t i) {
  return a.ids_i32 ? static_cast<const int32_t*>(a.targets)[i]
                   : static_cast<const int64_t*>(a.targets)[i];
}

// Counts the rows that are not ignored, and sets the words.  One block: it runs beside
// the rows' kernel (8,192 targets take it 3 us).
__global__ void __launch_bounds__(1024) loss_count_kernel(const __grid_constant__ LossArgs a) {
  __shared__ int32_t part[32];
  wait_for_predecessor();
  launch_dependents();
  int32_t n = 0;
  if (a.scale == nullptr)
    for (int64_t i = threadIdx.x; i < a.all_rows; i += 1024) n += target_of(a, i) != a.ignore;
  n = __reduce_add_sync(0xffffffffu, n);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    n = __reduce_add_sync(0xffffffffu, part[threadIdx.x]);
    if (threadIdx.x == 0) *a.words = Words{0, 0, n, n > 0 ? 1.0f / static_cast<float>(n) : 0.0f};
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int k = 16; k > 0; k /= 2) x += __shfl_xor_sync(0xffffffffu, x, k);
  return x;
}

// A warp a row: the target's logit, and x laid out for TMA, an ignored row's as zeros
// (its x may hold anything, and 0 times an infinity would reach dw).
template <bool VEC>
__global__ void __launch_bounds__(256) loss_rows_kernel(const __grid_constant__ LossArgs a) {
  // The first piece's rows do not wait for the count, whose kernel let this one begin when
  // all that came before was complete.
  if (a.first > 0) wait_for_predecessor();
  launch_dependents();
  const int lane = threadIdx.x % 32;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; i < a.rows;
       i += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t t = target_of(a, a.first + i);
    const bool ignored = t == a.ignore, column = !ignored && t >= 0 && t < a.vocab;
    const uint16_t* x = a.x + (a.first + i) * a.ldx;
    const uint16_t* w = a.w + (column ? t : 0) * a.ldw;
    uint16_t* to = a.xc + i * a.ldxc;
    float sum = 0.0f;
    if constexpr (VEC) {
      for (int64_t j = 8 * lane; j < a.width; j += 256) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (j + 8 <= a.width) {
          if (!ignored) v = *reinterpret_cast<const uint4*>(x + j);
          if (column) {
            float p[8], q[8];
            bf16x8(v, p);
            bf16x8(__ldg(reinterpret_cast<const uint4*>(w + j)), q);
#pragma unroll
            for (int c = 0; c < 8; ++c) sum = fmaf(p[c], q[c], sum);
          }
          *reinterpret_cast<uint4*>(to + j) = v;
        } else {
          for (int64_t k = j; k < a.width; ++k) {
            to[k] = ignored ? 0 : x[k];
            if (column) sum = fmaf(bf16_at(x + k), bf16_at(w + k), sum);
          }
        }
      }
    } else {
      for (int64_t j = lane; j < a.width; j += 32) {
        to[j] = ignored ? 0 : x[j];
        if (column) sum = fmaf(bf16_at(x + j), bf16_at(w + j), sum);
      }
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      const float zt = column || ignored ? sum : NAN;
      a.zt[i] = zt;
      a.ref[i] = isfinite(zt) ? zt : 0.0f;
      a.column[i] = column ? static_cast<int32_t>(t) : ignored ? -1 : -2;
    }
  }
  if (a.first == 0) wait_for_predecessor();
}

constexpr int kFinishThreads = 256, kFinishWarps = kFinishThreads / 32;

// A block a row: the row's sums in the order of its parts, its loss, and dz.  With c alike
// for all rows (the mean) dz is p less the target's 1, whose rounding is nothing where p is
// small, and c multiplies the products' sums; a scale of each row's own is in its dz.
// AGAIN: the second time, where the first has asked for it.  The last block adds up the
// losses.  Bound by HBM: 4 bytes an element (8192 x 50257: 1.65 GB).
template <bool AGAIN>
__global__ void __launch_bounds__(kFinishThreads) loss_finish_kernel(const __grid_constant__ LossArgs a) {
  __shared__ float2 part[kFinishWarps];
  __shared__ double sum_part[kFinishWarps];
  __shared__ int32_t last;
  wait_for_predecessor();
  launch_dependents();
  if (AGAIN && __ldcg(&a.words->again) == 0) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    const int32_t t = __ldcg(a.column + i);
    const float zt = __ldcg(a.zt + i), ref = __ldcg(a.ref + i);
    float sum = 0.0f, top = -INFINITY;
    if (t != -1) {
      for (int k = threadIdx.x; k < a.parts; k += kFinishThreads) {
        const float2 s = __ldcg(a.sums + i * a.parts + k);
        sum += s.x;
        top = fmaxf(top, s.y);
      }
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int k = 16; k > 0; k /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    __syncthreads();  // the row before is done with these
    if (lane == 0) part[warp] = make_float2(sum, top);
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kFinishWarps; ++k) {
      sum += part[k].x;
      top = fmaxf(top, part[k].y);
    }
    const bool own = zt == ref;
    const float et = own ? 1.0f : expf(zt - ref);
    const float whole = sum + et;
    float loss = own ? log1pf(sum) : (ref - zt) + logf(whole);
    // a NaN is no column's, or of the inputs'; an infinite logit leaves no gradient
    float f = (a.scale != nullptr ? __ldg(a.scale + a.first + i) : 1.0f) / whole;
    if (!isfinite(whole)) f = NAN;
    if (t == -1) loss = f = 0.0f;
    if (t == -2) loss = f = NAN;
    if (threadIdx.x == 0) {
      a.losses[a.first + i] = loss;
      if (!AGAIN && t >= 0 && sum > kOneMore && isfinite(top)) {
        a.ref[i] = top;
        a.words->again = 1;
      }
    }
    if (a.held == nullptr) continue;
    // (the pitch has room for whole vectors; an ignored row's are not read)
    uint16_t* row = a.held + i * a.ldz;
    constexpr int kSpan = 8 * kFinishThreads, U = 2;
    for (int64_t j0 = 8 * threadIdx.x; j0 < a.vocab; j0 += U * kSpan) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t != -1 && j0 + u * kSpan < a.vocab)
          v[u] = __ldcs(reinterpret_cast<const uint4*>(row + j0 + u * kSpan));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * kSpan;
        if (j >= a.vocab) break;
        float y[8] = {};
        if (t != -1) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int16_t d = static_cast<int16_t>(c % 2 ? w[c / 2] >> 16 : w[c / 2] & 0xffffu);
            const float e = fast_exp2(static_cast<float>(d) * (kLog2e / 1024.0f));
            y[c] = d == INT16_MIN ? f * 0.0f : f * e;
          }
          if (t - j >= 0 && t - j < 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (j + c == t) y[c] = -(f * sum);
          }
        }
        *reinterpret_cast<uint4*>(row + j) = to_bf16x8(y);
      }
    }
  }
  if (a.total == nullptr) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&a.words->ticket, 1) == static_cast<int32_t>(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (!AGAIN) {
    if (threadIdx.x == 0) a.words->ticket = 0;
    if (__ldcg(&a.words->again) != 0) return;  // there are other losses to come
  }
  // in 64 bits, a thread's own in chains of 8
  double total = 0.0;
  constexpr int U = 8;
  for (int64_t i0 = threadIdx.x; i0 < a.all_rows; i0 += U * kFinishThreads) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kFinishThreads;
      x[u] = i < a.all_rows ? __ldcg(a.losses + i) : 0.0f;
      if (a.scale != nullptr && i < a.all_rows && target_of(a, i) != a.ignore)
        total += static_cast<double>(__ldg(a.scale + i)) * static_cast<double>(x[u]);
    }
    if (a.scale == nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u) total += static_cast<double>(x[u]);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k /= 2) total += __shfl_xor_sync(0xffffffffu, total, k);
  if (lane == 0) sum_part[warp] = total;
  __syncthreads();
  if (threadIdx.x != 0) return;
  total = 0.0;
  for (int k = 0; k < kFinishWarps; ++k) total += sum_part[k];
  if (a.scale == nullptr) {
    const int32_t valid = __ldcg(&a.words->valid);
    total = valid > 0 ? total / valid : 0.0;
  }
  *a.total = static_cast<float>(total);
}

// The next piece of rows asks anew.
__global__ void loss_next_kernel(Words* words) {
  wait_for_predecessor();
  launch_dependents();
  words->again = 0;
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
  const int64_t row = grads ? 2 * laid_out_pitch(s.vocab) : 16;
  int64_t n = kMostHeld / row / 256 * 256;
  if (n < 256) n = 256;
  return s.rows < n ? s.rows : n;
}

// Where a call's arrays lie in its workspace.
struct Layout {
  int64_t piece, parts;  // rows of a piece, and parts of the vocabulary at most
  int64_t w, x, zt, held, sums, losses, acc, linear, bytes;
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
  l.x = take(2 * l.piece * laid_out_pitch(s.width));
  l.zt = take(12 * l.piece);  // zt, ref, column
  l.held = take(grads ? 2 * l.piece * laid_out_pitch(s.vocab) : 0);
  l.sums = take(8 * l.piece * l.parts);
  l.losses = take(4 * s.rows);
  const bool sums32 = grads && s.rows > l.piece && (flags & ZERO_GRAD_F32) == 0;
  l.acc = take(sums32 ? 4 * s.vocab * round_up(s.width, 4) : 0);
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
  a.xc = reinterpret_cast<uint16_t*>(base + l.x);
  a.ldxc = laid_out_pitch(s.width);
  a.sums = reinterpret_cast<const float2*>(base + l.sums);
  a.scale = L.scale;
  a.losses = L.losses != nullptr ? L.losses : reinterpret_cast<float*>(base + l.losses);
  a.held = grads ? reinterpret_cast<uint16_t*>(base + l.held) : nullptr;
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
  if (e == cudaSuccess) e = chain.launch(loss_count_kernel, dim3(1), 1024, 0, 1, a);
  const bool joined = L.dw != nullptr && s.rows > l.piece && !L.grad_f32;  // sums of pieces in fp32
  float* acc = reinterpret_cast<float*>(base + l.acc);
  const auto blocks_of = [](int64_t n, int64_t most) {
    return dim3(static_cast<unsigned>(n < most ? n : most));
  };
  for (int64_t first = 0; e == cudaSuccess && first < s.rows; first += l.piece) {
    a.first = first;
    a.rows = s.rows - first < l.piece ? s.rows - first : l.piece;
    const bool last = first + a.rows == s.rows;
    a.parts = static_cast<int32_t>(exponent_parts(a.rows, s.vocab, s.width));
    a.total = last ? L.total : nullptr;
    if (first > 0) e = chain.launch(loss_next_kernel, dim3(1), 1, 0, 1, a.words);
    if (e == cudaSuccess)
      e = chain.launch(a.vec ? loss_rows_kernel<true> : loss_rows_kernel<false>,
                       blocks_of((a.rows + 7) / 8, 16 * kSms), 256, 0, 1, a);
    ExponentLaunch x{};
    x.rows = a.rows;
    x.width = s.width;
    x.vocab = s.vocab;
    x.x = a.xc;
    x.ldx = a.ldxc;
    x.w = w;
    x.ldw = ldw;
    x.of = {a.ref, a.column, const_cast<float2*>(a.sums), a.parts, nullptr};
    x.out = a.held;
    x.ldo = a.ldz;
    x.stream = L.stream;
    x.withhold = L.withhold;
    if (e == cudaSuccess) e = launch_exponents(x);
    const dim3 grid = blocks_of(a.rows, 8 * kSms);
    if (e == cudaSuccess) e = chain.launch(loss_finish_kernel<false>, grid, kFinishThreads, 0, 1, a);
    x.of.only_if = &a.words->again;
    if (e == cudaSuccess) e = launch_exponents(x);
    if (e == cudaSuccess)
      e = chain.launch(loss_finish_kernel<true>, blocks_of(a.rows, 2 * kSms), kFinishThreads, 0, 1, a);
    if (e != cudaSuccess || !grads) continue;
    LinearBackwardLaunch b{};
    b.s = linear_of(s, a.rows);
    b.s.ldw = ldw;
    b.dy = a.held;
    b.x = a.xc;
    b.w = w;
    b.dx = L.dx != nullptr ? L.dx + first * s.lddx : nullptr;
    b.dw = joined ? acc : L.dw;
    if (joined) b.s.lddw = round_up(s.width, 4);
    b.grad_f32 = L.grad_f32 || joined;
    b.accumulate = first > 0 || (L.accumulate && !joined);
    b.scale = L.scale == nullptr ? &a.words->share : nullptr;
    b.workspace = base + l.linear;
    b.stream = L.stream;
    b.withhold = L.withhold;
    e = launch_linear_backward(b);
  }
  if (e == cudaSuccess && joined)
    e = chain.launch(loss_round_kernel, blocks_of(s.vocab, 16 * kSms), 256, 0, 1, acc,
                     round_up(s.width, 4), static_cast<uint16_t*>(L.dw), s.lddw, s.vocab, s.width,
                     L.accumulate);
  return e;
}

}  // namespace zeroadam
