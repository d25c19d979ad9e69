// embedding.cu -- rows of a table looked up by token ids, and the gradient of the
// table, on sm_103a.
#include "chain.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

__device__ __forceinline__ int64_t id_at(const void* ids, int32_t i32, int64_t i) {
  return i32 ? __ldg(static_cast<const int32_t*>(ids) + i)
             : __ldg(static_cast<const long long*>(ids) + i);
}

// ------------------------------------------------------------------------ forward

struct LookupArgs {
  const uint16_t* table;
  const void* ids;
  uint16_t* y;
  int64_t rows, width, vocab, ldt, ldy;
  int64_t spans;   // of kSpan columns a row has
  int32_t ids_i32;
  float scale;
};

constexpr int kVectors = 4, kSpan = 256 * kVectors;  // columns of a warp's item

// y = scale * table[id]: a warp takes 1,024 columns of a row, four 16-byte vectors a
// lane, all asked for before the first is used.  Bound by HBM.
template <bool VEC>
__global__ void __launch_bounds__(256) embedding_lookup_kernel(const __grid_constant__ LookupArgs a) {
  wait_for_predecessor();
  launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t items = a.rows * a.spans;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; q < items;
       q += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t i = q / a.spans, j0 = (q - i * a.spans) * kSpan;
    const int64_t id = id_at(a.ids, a.ids_i32, i);
    const bool known = id >= 0 && id < a.vocab;
    const uint16_t* from = a.table + (known ? id : 0) * a.ldt;
    uint16_t* to = a.y + i * a.ldy;
    const float scale = known ? a.scale : NAN;
    if constexpr (VEC) {
      uint4 v[kVectors];
#pragma unroll
      for (int k = 0; k < kVectors; ++k) {
        const int64_t j = j0 + 256 * k + 8 * lane;
        v[k] = known && j + 8 <= a.width ? __ldg(reinterpret_cast<const uint4*>(from + j))
                                         : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kVectors; ++k) {
        const int64_t j = j0 + 256 * k + 8 * lane;
        if (j + 8 <= a.width) {
          float x[8];
          bf16x8(v[k], x);
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] *= scale;
          *reinterpret_cast<uint4*>(to + j) = to_bf16x8(x);
        } else {
          for (int64_t c = j; c < a.width; ++c) to[c] = to_bf16(known ? bf16_at(from + c) * scale : NAN);
        }
      }
    } else {
#pragma unroll 8
      for (int k = 0; k < kSpan / 32; ++k) {
        const int64_t j = j0 + 32 * k + lane;
        if (j < a.width) to[j] = to_bf16(known ? bf16_at(from + j) * scale : NAN);
      }
    }
  }
}

// ----------------------------------------------------------------------- backward
//
// dtable[v] = scale * sum of dy[i] over the rows i with id v.  The tokens are dealt out to
// `classes` classes, v going to class v mod classes, so that the commonest ones, which
// lie together in most vocabularies, fall to different ones; and the columns to slices of
// 256.  A block takes one class and one slice, and needs nothing of any other: it finds
// its class's rows among the ids (which all blocks read, from L2), sorts them by token,
// keeping the rows' order, sums each token's rows in registers, and writes every row of
// its class, zeros where no token was.  Neither sums nor places go through atomics on
// floats or other blocks, so the result follows from the ids alone.

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kSlice = 256;      // columns: 8 a lane
constexpr int kWindow = 4096;    // tokens of a class that are sorted at one time
constexpr int kMostRows = 6144;  // rows that are sorted at one time
constexpr int kEachRows = kMostRows / kSumWarps;
constexpr int kOneWarp = 48;     // rows of a token that one warp sums by itself

struct ScatterArgs {
  const uint16_t* dy;
  const void* ids;
  void* dtable;
  int64_t rows, width, vocab, ldy, ldt, padding;
  int32_t ids_i32, grad_f32, accumulate;
  int32_t classes;
  float scale;
};

struct ScatterShared {
  int32_t offset[kWindow + 1];  // counts; then where a token's rows begin; then where they end
  int32_t row[kMostRows];       // the class's rows in their order, kEachRows for each warp
  uint16_t token[kMostRows];    // and their tokens, within the window
  int32_t sorted[kMostRows];    // rows by token
  uint16_t some[kWindow];       // tokens that have rows
  float part[kSumWarps][kSlice];
  int32_t found[kSumWarps];     // rows of each warp
  int32_t scan[2][kSumWarps];
  int32_t next_sum, next_zero;  // items taken
};

// The sum of a run of rows: 8 columns a lane, in the order of the rows, eight rows' loads
// under way at a time.  A chain ends after 64 rows, so that its error does not grow with
// a common token's count.
template <bool VEC>
struct SliceSum {
  float run[8] = {}, sum[8] = {};
  int chain = 0;

  __device__ __forceinline__ void add(const ScatterArgs& a, const int32_t* rows, int n, int64_t col,
                                      int lane) {
    constexpr int U = 8;
#pragma unroll 1
    for (int k = 0; k < n; k += U) {
      if constexpr (VEC) {
        uint4 v[U];
        const bool in = col + 8 * lane + 8 <= a.width;
        const uint16_t* from = a.dy + col + 8 * lane;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          v[u] = make_uint4(0, 0, 0, 0);
          if (k + u < n && in) v[u] = __ldg(reinterpret_cast<const uint4*>(from + rows[k + u] * a.ldy));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[8];
          bf16x8(v[u], x);
#pragma unroll
          for (int c = 0; c < 8; ++c) run[c] += x[c];
        }
        if (!in && col + 8 * lane < a.width) {
#pragma unroll 1
          for (int u = 0; u < U && k + u < n; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (col + 8 * lane + c < a.width) run[c] += bf16_at(from + rows[k + u] * a.ldy + c);
        }
      } else {
#pragma unroll
        for (int h = 0; h < U; h += 2) {
          float x[2][8];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int64_t j = col + lane + 32 * c;
              x[u][c] = k + h + u < n && j < a.width ? bf16_at(a.dy + rows[k + h + u] * a.ldy + j) : 0.0f;
            }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c) run[c] += x[u][c];
        }
      }
      if ((chain += U) >= 64) join();
    }
  }
  __device__ __forceinline__ void join() {
    chain = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      sum[c] += run[c];
      run[c] = 0.0f;
    }
  }
};

// A lane's 8 columns of one row of the table's gradient.
template <bool VEC>
__device__ __forceinline__ void put_slice(const ScatterArgs& a, int64_t v, int64_t col, const float x[8],
                                          int lane) {
  const int64_t at = v * a.ldt + col;
  if (VEC && col + 8 * lane + 8 <= a.width) {
    if (a.grad_f32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.dtable) + at + 8 * lane);
      float4 p = make_float4(0, 0, 0, 0), q = p;
      if (a.accumulate) {
        p = o[0];
        q = o[1];
      }
      o[0] = make_float4(p.x + x[0], p.y + x[1], p.z + x[2], p.w + x[3]);
      o[1] = make_float4(q.x + x[4], q.y + x[5], q.z + x[6], q.w + x[7]);
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dtable) + at + 8 * lane);
      float y[8] = {};
      if (a.accumulate) bf16x8(*o, y);
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] += x[c];
      *o = to_bf16x8(y);
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int64_t j = VEC ? 8 * lane + c : lane + 32 * c;
    if (col + j >= a.width) continue;
    if (a.grad_f32) {
      float* o = static_cast<float*>(a.dtable) + at + j;
      *o = a.accumulate ? *o + x[c] : x[c];
    } else {
      uint16_t* o = static_cast<uint16_t*>(a.dtable) + at + j;
      *o = to_bf16(a.accumulate ? bf16_at(o) + x[c] : x[c]);
    }
  }
}

// A block's place: its class, its slice, and the window of tokens under way.
struct ScatterPlace {
  int64_t col, w0;
  uint32_t mine, classes;
  int window;
  // row i's token within the window, or -1
  __device__ __forceinline__ int token_of(const ScatterArgs& a, int64_t i) const {
    const int64_t id = id_at(a.ids, a.ids_i32, i);
    const uint32_t k = static_cast<uint32_t>(id) / classes;
    const int64_t t = static_cast<int64_t>(k) - w0;
    const bool good = id >= 0 && id < a.vocab && id != a.padding &&
                      static_cast<uint32_t>(id) - k * classes == mine && t >= 0 && t < window;
    return good ? static_cast<int>(t) : -1;
  }
};

// The sum of a token's rows, scaled and written.
template <bool VEC>
__device__ __forceinline__ void finish_token(const ScatterArgs& a, const ScatterPlace& p, SliceSum<VEC>& s,
                                             int t, int lane) {
  s.join();
#pragma unroll
  for (int c = 0; c < 8; ++c) s.sum[c] *= a.scale;
  put_slice<VEC>(a, (p.w0 + t) * p.classes + p.mine, p.col, s.sum, lane);
}

// n rows by the whole block: a run of them a warp, the warps' sums added in their order.
template <bool VEC>
__device__ __forceinline__ void finish_token_together(const ScatterArgs& a, const ScatterPlace& p,
                                                      ScatterShared& sh, SliceSum<VEC>& s, int t) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  s.join();
#pragma unroll
  for (int c = 0; c < 8; ++c) sh.part[warp][32 * c + lane] = s.sum[c];
  __syncthreads();
  if (warp == 0) {
    for (int k = 1; k < kSumWarps; ++k)
#pragma unroll
      for (int c = 0; c < 8; ++c) s.sum[c] += sh.part[k][32 * c + lane];
    finish_token(a, p, s, t, lane);
  }
  __syncthreads();
}
template <bool VEC>
__device__ __forceinline__ void add_share(const ScatterArgs& a, const ScatterPlace& p, SliceSum<VEC>& s,
                                          const int32_t* rows, int n) {
  const int warp = threadIdx.x / 32, per = (n + kSumWarps - 1) / kSumWarps;
  const int first = warp * per < n ? warp * per : n, end = first + per < n ? first + per : n;
  s.add(a, rows + first, end - first, p.col, threadIdx.x % 32);
}

// Rows [i0, i1) of tokens [t0, t1) in their order, each warp's own run of rows in its own
// part of the list; whether all have room.  (All threads; found[] can be read after it.)
__device__ __forceinline__ bool list_rows(const ScatterArgs& a, const ScatterPlace& p, ScatterShared& sh,
                                          int64_t i0, int64_t i1, int t0, int t1, bool count) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t each = (i1 - i0 + kSumThreads - 1) / kSumThreads * 32;
  const int64_t from = i0 + warp * each, to = from + each < i1 ? from + each : i1;
  int n = 0;
  constexpr int U = 8;
  for (int64_t i = from; i < to; i += 32 * U) {
    int t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = i + 32 * u + lane < to ? p.token_of(a, i + 32 * u + lane) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool has = t[u] >= t0 && t[u] < t1;
      const uint32_t all = __ballot_sync(0xffffffffu, has);
      if (has) {
        const int at = n + __popc(all & ((1u << lane) - 1u));
        if (at < kEachRows) {
          sh.row[warp * kEachRows + at] = static_cast<int32_t>(i + 32 * u + lane);
          sh.token[warp * kEachRows + at] = static_cast<uint16_t>(t[u]);
        }
        if (count) atomicAdd(&sh.offset[t[u]], 1);
      }
      n += __popc(all);
    }
  }
  if (lane == 0) sh.found[warp] = n;
  return __syncthreads_and(n <= kEachRows) != 0;
}

// The listed rows by token, each token's in the order of the list: a warp takes every 8th
// token.  sorted[offset[t] - start ...], and offset[t] becomes the end.
__device__ __forceinline__ void sort_rows(ScatterShared& sh, int start) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int w = 0; w < kSumWarps; ++w) {
    const int n = sh.found[w];
    for (int k = 0; k < n; k += 32) {
      const int t = k + lane < n ? sh.token[w * kEachRows + k + lane] : -1;
      const bool take = t >= 0 && t % kSumWarps == warp;
      const uint32_t takers = __ballot_sync(0xffffffffu, take);
      if (take) {
        const uint32_t same = __match_any_sync(takers, t);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int at = sh.offset[t];
        sh.sorted[at - start + before] = sh.row[w * kEachRows + k + lane];
        __syncwarp(takers);
        if (before == 0) sh.offset[t] = at + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
}

// The next item of a kind, for a warp.
__device__ __forceinline__ int take_item(int32_t* next, int lane) {
  int k = 0;
  if (lane == 0) k = atomicAdd(next, 1);
  return __shfl_sync(0xffffffffu, k, 0);
}

template <bool VEC>
__global__ void __launch_bounds__(kSumThreads, 2)
    embedding_scatter_kernel(const __grid_constant__ ScatterArgs a) {
  extern __shared__ uint8_t raw[];
  ScatterShared& sh = *reinterpret_cast<ScatterShared*>(raw);
  wait_for_predecessor();
  launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  ScatterPlace p;
  p.col = static_cast<int64_t>(blockIdx.y) * kSlice;
  p.mine = blockIdx.x;
  p.classes = a.classes;
  const int64_t tokens = (a.vocab - p.mine + p.classes - 1) / p.classes;  // of this class

  for (p.w0 = 0; p.w0 < tokens; p.w0 += kWindow) {
    const int window = tokens - p.w0 < kWindow ? static_cast<int>(tokens - p.w0) : kWindow;
    p.window = window;
    for (int t = threadIdx.x; t <= window; t += kSumThreads) sh.offset[t] = 0;
    if (threadIdx.x == 0) sh.next_sum = sh.next_zero = 0;
    __syncthreads();
    const bool room = list_rows(a, p, sh, 0, a.rows, 0, window, true);
    // counts to offsets, and the tokens that have rows: a thread takes a run of tokens
    int some = 0;
    {
      const int per = (window + kSumThreads - 1) / kSumThreads;
      const int t0 = threadIdx.x * per < window ? threadIdx.x * per : window;
      const int t1 = t0 + per < window ? t0 + per : window;
      int rows = 0;
      for (int t = t0; t < t1; ++t) {
        rows += sh.offset[t];
        some += sh.offset[t] > 0;
      }
      int x = rows, y = some;
#pragma unroll
      for (int k = 1; k < 32; k *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, x, k), v = __shfl_up_sync(0xffffffffu, y, k);
        if (lane >= k) {
          x += u;
          y += v;
        }
      }
      if (lane == 31) {
        sh.scan[0][warp] = x;
        sh.scan[1][warp] = y;
      }
      __syncthreads();
      int before = x - rows, at = y - some, all = 0;
      some = 0;
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w) {
        if (w < warp) {
          before += sh.scan[0][w];
          at += sh.scan[1][w];
        }
        all += sh.scan[0][w];
        some += sh.scan[1][w];
      }
      for (int t = t0; t < t1; ++t) {
        const int n = sh.offset[t];
        sh.offset[t] = before;
        before += n;
        if (n > 0) sh.some[at++] = static_cast<uint16_t>(t);
      }
      if (threadIdx.x == 0) sh.offset[window] = all;
      __syncthreads();
    }
    // tokens of no row: zeros
    const int zeros = a.accumulate ? 0 : (window + 31) / 32;
    const auto zero_item = [&](int k, bool sorted) {
      const int t = 32 * k + lane;
      bool none = false;
      if (t < window)
        none = sorted ? (t == 0 ? 0 : sh.offset[t - 1]) == sh.offset[t] : sh.offset[t] == sh.offset[t + 1];
      uint32_t left = __ballot_sync(0xffffffffu, none);
      const float zero[8] = {};
      while (left != 0) {
        const int u = __ffs(left) - 1;
        left &= left - 1;
        put_slice<VEC>(a, (p.w0 + 32 * k + u) * p.classes + p.mine, p.col, zero, lane);
      }
    };
    if (room) {
      sort_rows(sh, 0);
      const auto begin_of = [&](int t) { return t == 0 ? 0 : sh.offset[t - 1]; };
      // Half of the warps begin with the zeros, which fill the way to memory, half with
      // the sums, which wait for it.
      const auto sums = [&] {
        for (int k; (k = take_item(&sh.next_sum, lane)) < some;) {
          const int t = sh.some[k], first = begin_of(t), n = sh.offset[t] - first;
          if (n > kOneWarp) continue;
          SliceSum<VEC> s;
          s.add(a, sh.sorted + first, n, p.col, lane);
          finish_token(a, p, s, t, lane);
        }
      };
      if (warp % 2 == 0) sums();
      for (int k; (k = take_item(&sh.next_zero, lane)) < zeros;) zero_item(k, true);
      if (warp % 2 != 0) sums();
      for (int k0 = 0; k0 < some; k0 += 32) {
        const int k = k0 + lane, mine = k < some ? sh.some[k] : 0;
        uint32_t left = __ballot_sync(0xffffffffu, k < some && sh.offset[mine] - begin_of(mine) > kOneWarp);
        while (left != 0) {  // alike in every warp
          const int t = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
          left &= left - 1;
          const int first = begin_of(t);
          SliceSum<VEC> s;
          add_share(a, p, s, sh.sorted + first, sh.offset[t] - first);
          finish_token_together(a, p, sh, s, t);
        }
      }
      __syncthreads();
      continue;
    }
    // More rows than there is room for: tokens from t0 up to t1, as many as fit however
    // they lie; a token of more rows than that goes alone, its rows in runs.  The ids are
    // read once more for each.
    for (int k = warp; k < zeros; k += kSumWarps) zero_item(k, false);
    __syncthreads();
    for (int t0 = 0; t0 < window;) {
      const int start = sh.offset[t0];
      int lo = t0 + 1, hi = window;  // the last t1 whose rows have room, or t0 + 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (sh.offset[mid] - start <= kEachRows) lo = mid;
        else hi = mid - 1;
      }
      const int t1 = lo, count = sh.offset[t1] - start;
      __syncthreads();
      if (count > kEachRows) {
        SliceSum<VEC> s;
        for (int64_t i0 = 0; i0 < a.rows; i0 += kMostRows) {
          const int64_t i1 = i0 + kMostRows < a.rows ? i0 + kMostRows : a.rows;
          list_rows(a, p, sh, i0, i1, t0, t1, false);  // (a warp looks at kEachRows rows)
          s.add(a, sh.row + warp * kEachRows, sh.found[warp], p.col, lane);
          __syncthreads();
        }
        finish_token_together(a, p, sh, s, t0);
      } else if (count > 0) {
        list_rows(a, p, sh, 0, a.rows, t0, t1, false);
        sort_rows(sh, start);
        for (int t = t0; t < t1; ++t) {
          const int first = (t == t0 ? start : sh.offset[t - 1]), n = sh.offset[t] - first;
          if (n == 0 || (n <= kOneWarp && t % kSumWarps != warp)) continue;
          SliceSum<VEC> s;
          if (n <= kOneWarp) {
            s.add(a, sh.sorted + first - start, n, p.col, lane);
            finish_token(a, p, s, t, lane);
          } else {
            add_share(a, p, s, sh.sorted + first - start, n);
            finish_token_together(a, p, sh, s, t);
          }
        }
        __syncthreads();
      }
      t0 = t1;
    }
  }
}

template <bool VEC>
cudaError_t launch_scatter(const ScatterArgs& a, Chain* chain) {
  constexpr int smem = static_cast<int>(sizeof(ScatterShared));
  static_assert(smem <= 113 * 1024, "two blocks an SM");
  const auto kernel = embedding_scatter_kernel<VEC>;
  // (a property of the kernel on the current device, set alike by every call)
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t slices = (a.width + kSlice - 1) / kSlice;
  for (int64_t k = 0; k < slices; k += 65535) {  // the grid's y side ends there
    ScatterArgs part = a;
    part.dy += k * kSlice;
    part.dtable = a.grad_f32 ? static_cast<void*>(static_cast<float*>(a.dtable) + k * kSlice)
                             : static_cast<void*>(static_cast<uint16_t*>(a.dtable) + k * kSlice);
    part.width -= k * kSlice;
    const int64_t high = slices - k < 65535 ? slices - k : 65535;
    const cudaError_t e2 = chain->launch(kernel, dim3(a.classes, static_cast<unsigned>(high)),
                                         kSumThreads, smem, 1, part);
    if (e2 != cudaSuccess) return e2;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_embedding_forward(const EmbeddingLaunch& L) {
  (void)cudaGetLastError();
  const zero_embedding_t& s = L.s;
  LookupArgs a{};
  a.table = L.from;
  a.ids = L.ids;
  a.y = static_cast<uint16_t*>(L.to);
  a.rows = s.rows;
  a.width = s.width;
  a.vocab = s.vocab;
  a.ldt = s.ldt;
  a.ldy = s.ldy;
  a.spans = (s.width + kSpan - 1) / kSpan;
  a.ids_i32 = L.ids_i32;
  a.scale = L.scale;
  const bool vec = aligned(L.from, 16) && aligned(L.to, 16) && (s.vocab == 1 || s.ldt % 8 == 0) &&
                   (s.rows == 1 || s.ldy % 8 == 0);
  const int64_t blocks = (s.rows * a.spans + 7) / 8;
  Chain chain{L.stream};
  return chain.launch(vec ? embedding_lookup_kernel<true> : embedding_lookup_kernel<false>,
                      dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), 256, 0, 1, a);
}

cudaError_t launch_embedding_backward(const EmbeddingLaunch& L) {
  (void)cudaGetLastError();
  const zero_embedding_t& s = L.s;
  ScatterArgs a{};
  a.dy = L.from;
  a.ids = L.ids;
  a.dtable = L.to;
  a.rows = s.rows;
  a.width = s.width;
  a.vocab = s.vocab;
  a.ldy = s.ldy;
  a.ldt = s.ldt;
  a.padding = L.padding;
  a.ids_i32 = L.ids_i32;
  a.grad_f32 = L.grad_f32;
  a.accumulate = L.accumulate;
  a.scale = L.scale;
  // two blocks an SM in all; more where a class would have over half of the rows that a
  // block has room for
  const int64_t slices = (s.width + kSlice - 1) / kSlice;
  int64_t classes = 2 * kSms / slices;
  const int64_t least = s.rows / (kMostRows / 2) + 1;
  if (classes < least) classes = least;
  a.classes = static_cast<int32_t>(classes < s.vocab ? classes : s.vocab);
  const bool vec = aligned(L.from, 16) && aligned(L.to, 16) && (s.rows == 1 || s.ldy % 8 == 0) &&
                   (s.vocab == 1 || s.ldt % (L.grad_f32 ? 4 : 8) == 0);
  Chain chain{L.stream};
  return vec ? launch_scatter<true>(a, &chain) : launch_scatter<false>(a, &chain);
}

}  // namespace zeroadam
