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
  int32_t offset[kWindow + 1];       // counts, then where each token's rows begin
  int32_t cursor[kWindow];           // where the next one goes
  int32_t row[kMostRows];            // the class's rows in their order
  uint16_t token[kMostRows];         // and their tokens, within the window
  int32_t sorted[kMostRows];         // rows by token
  float part[kSumWarps][kSlice];
  int32_t warp_count[kSumWarps + 1];
  int32_t found;
};

// The sum of a run of rows: 8 columns a lane, in the order of the rows, four rows' loads
// under way at a time.  A chain ends after 64 rows, so that its error does not grow with
// a common token's count.
template <bool VEC>
struct SliceSum {
  float run[8] = {}, sum[8] = {};
  int chain = 0;

  __device__ __forceinline__ void add(const ScatterArgs& a, const int32_t* rows, int n, int64_t col,
                                      int lane) {
    for (int k = 0; k < n; k += 4) {
      float x[4][8];
      if constexpr (VEC) {
        uint4 v[4];
        const bool in = col + 8 * lane + 8 <= a.width;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = make_uint4(0, 0, 0, 0);
          if (k + u < n && in)
            v[u] = __ldg(reinterpret_cast<const uint4*>(a.dy + rows[k + u] * a.ldy + col + 8 * lane));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          bf16x8(v[u], x[u]);
          if (!in && k + u < n) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (col + 8 * lane + c < a.width)
                x[u][c] = bf16_at(a.dy + rows[k + u] * a.ldy + col + 8 * lane + c);
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int64_t j = col + lane + 32 * c;
            x[u][c] = k + u < n && j < a.width ? bf16_at(a.dy + rows[k + u] * a.ldy + j) : 0.0f;
          }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int c = 0; c < 8; ++c) run[c] += x[u][c];
      if ((chain += 4) >= 64) join();
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

template <bool VEC>
__global__ void __launch_bounds__(kSumThreads, 2)
    embedding_scatter_kernel(const __grid_constant__ ScatterArgs a) {
  extern __shared__ uint8_t raw[];
  ScatterShared& sh = *reinterpret_cast<ScatterShared*>(raw);
  wait_for_predecessor();
  launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * kSlice;
  const int64_t mine = blockIdx.x, classes = a.classes;
  const int64_t tokens = (a.vocab - mine + classes - 1) / classes;  // of this class

  for (int64_t w0 = 0; w0 < tokens; w0 += kWindow) {
    const int window = tokens - w0 < kWindow ? static_cast<int>(tokens - w0) : kWindow;
    // row i's token within the window, or -1
    const auto token_of = [&](int64_t i) {
      const int64_t id = id_at(a.ids, a.ids_i32, i);
      if (id < 0 || id >= a.vocab || id == a.padding) return -1;
      const uint32_t k = static_cast<uint32_t>(id) / static_cast<uint32_t>(classes);
      if (static_cast<uint32_t>(id) - k * static_cast<uint32_t>(classes) != static_cast<uint32_t>(mine))
        return -1;
      const int64_t t = static_cast<int64_t>(k) - w0;
      return t >= 0 && t < window ? static_cast<int>(t) : -1;
    };
    __syncthreads();
    for (int t = threadIdx.x; t <= window; t += kSumThreads) sh.offset[t] = 0;
    __syncthreads();
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < a.rows; i += kSumThreads) {
      const int t = token_of(i);
      if (t >= 0) atomicAdd(&sh.offset[t], 1);
    }
    __syncthreads();
    // rows of no token: zeros, on their way while the others are sorted
    if (!a.accumulate) {
      const float zero[8] = {};
      for (int t = warp; t < window; t += kSumWarps)
        if (sh.offset[t] == 0) put_slice<VEC>(a, (w0 + t) * classes + mine, col, zero, lane);
    }
    __syncthreads();
    // counts to offsets
    if (warp == 0) {
      int base = 0;
      for (int t0 = 0; t0 < window; t0 += 32) {
        const int n = t0 + lane < window ? sh.offset[t0 + lane] : 0;
        int run = n;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, run, k);
          if (lane >= k) run += y;
        }
        if (t0 + lane < window) sh.offset[t0 + lane] = base + run - n;
        base += __shfl_sync(0xffffffffu, run, 31);
      }
      if (lane == 0) sh.offset[window] = base;
    }
    __syncthreads();
    // tokens from t0 up to t1, as many as there is room for; a token of more rows than
    // that goes alone, its rows in as many runs as it takes
    for (int t0 = 0; t0 < window;) {
      int t1 = window;
      if (sh.offset[window] - sh.offset[t0] > kMostRows) {
        int lo = t0 + 1, hi = window;  // the last t1 whose rows have room, or t0 + 1
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (sh.offset[mid] - sh.offset[t0] <= kMostRows) lo = mid;
          else hi = mid - 1;
        }
        t1 = lo;
      }
      const int count = sh.offset[t1] - sh.offset[t0];
      if (count == 0) {
        t0 = t1;
        continue;
      }
      const bool alone = count > kMostRows;
      SliceSum<VEC> long_sum;  // of a token that goes alone: this warp's share
      for (int64_t i0 = 0; i0 < a.rows; i0 += alone ? kMostRows : a.rows) {
        const int64_t i1 = alone && i0 + kMostRows < a.rows ? i0 + kMostRows : a.rows;
        // the rows of these tokens in their order: a warp looks through a run of rows,
        // once to count and once to write
        const int64_t each = (i1 - i0 + kSumThreads - 1) / kSumThreads * 32;
        const int64_t from = i0 + warp * each, to = from + each < i1 ? from + each : i1;
        const auto in_range = [&](int64_t i) {
          const int t = i < to ? token_of(i) : -1;
          return t >= t0 && t < t1 ? t : -1;
        };
        int n = 0;
#pragma unroll 4
        for (int64_t i = from; i < to; i += 32)
          n += __popc(__ballot_sync(0xffffffffu, in_range(i + lane) >= 0));
        __syncthreads();
        if (lane == 0) sh.warp_count[warp] = n;
        __syncthreads();
        int base = 0, found = 0;
#pragma unroll
        for (int k = 0; k < kSumWarps; ++k) {
          const int c = sh.warp_count[k];
          if (k < warp) base += c;
          found += c;
        }
#pragma unroll 4
        for (int64_t i = from; i < to; i += 32) {
          const int t = in_range(i + lane);
          const uint32_t has = __ballot_sync(0xffffffffu, t >= 0);
          if (t >= 0) {
            const int at = base + __popc(has & ((1u << lane) - 1u));
            sh.row[at] = static_cast<int32_t>(i + lane);
            sh.token[at] = static_cast<uint16_t>(t);
          }
          base += __popc(has);
        }
        __syncthreads();
        if (alone) {
          // all of them are the token's: a run of rows a warp
          const int per = (found + kSumWarps - 1) / kSumWarps;
          const int first = warp * per < found ? warp * per : found;
          const int end = first + per < found ? first + per : found;
          long_sum.add(a, sh.row + first, end - first, col, lane);
          __syncthreads();
          continue;
        }
        // by token: a warp takes every 8th token, and its rows as they come
        for (int t = t0 + threadIdx.x; t < t1; t += kSumThreads)
          sh.cursor[t] = sh.offset[t] - sh.offset[t0];
        __syncthreads();
        for (int k = 0; k < found; k += 32) {
          const int t = k + lane < found ? sh.token[k + lane] : -1;
          const bool take = t >= 0 && t % kSumWarps == warp;
          const uint32_t takers = __ballot_sync(0xffffffffu, take);
          if (take) {
            const uint32_t same = __match_any_sync(takers, t);
            const int before = __popc(same & ((1u << lane) - 1u));
            const int at = sh.cursor[t];
            sh.sorted[at + before] = sh.row[k + lane];
            __syncwarp(takers);
            if (before == 0) sh.cursor[t] = at + __popc(same);
          }
          __syncwarp();
        }
        __syncthreads();
      }
      const auto finish = [&](SliceSum<VEC>& s, int t) {
        s.join();
#pragma unroll
        for (int c = 0; c < 8; ++c) s.sum[c] *= a.scale;
        put_slice<VEC>(a, (w0 + t) * classes + mine, col, s.sum, lane);
      };
      // the 8 warps' shares of a token, added up in their order by the first
      const auto join_warps = [&](SliceSum<VEC>& s, int t) {
        s.join();
#pragma unroll
        for (int c = 0; c < 8; ++c) sh.part[warp][32 * c + lane] = s.sum[c];
        __syncthreads();
        if (warp == 0) {
          for (int k = 1; k < kSumWarps; ++k)
#pragma unroll
            for (int c = 0; c < 8; ++c) s.sum[c] += sh.part[k][32 * c + lane];
          finish(s, t);
        }
        __syncthreads();
      };
      if (alone) {
        join_warps(long_sum, t0);
      } else {
        const int32_t start = sh.offset[t0];
        for (int t = t0 + warp; t < t1; t += kSumWarps) {
          const int first = sh.offset[t] - start, n = sh.offset[t + 1] - sh.offset[t];
          if (n == 0 || n > kOneWarp) continue;
          SliceSum<VEC> s;
          s.add(a, sh.sorted + first, n, col, lane);
          finish(s, t);
        }
        for (int t = t0; t < t1; ++t) {
          const int first = sh.offset[t] - start, n = sh.offset[t + 1] - sh.offset[t];
          if (n <= kOneWarp) continue;
          const int per = (n + kSumWarps - 1) / kSumWarps;
          const int begin = warp * per < n ? warp * per : n, end = begin + per < n ? begin + per : n;
          SliceSum<VEC> s;
          s.add(a, sh.sorted + first + begin, end - begin, col, lane);
          join_warps(s, t);
        }
      }
      __syncthreads();
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
  // two blocks an SM in all, at least one class
  const int64_t slices = (s.width + kSlice - 1) / kSlice;
  int64_t classes = 2 * kSms / slices;
  if (classes < 1) classes = 1;
  a.classes = static_cast<int32_t>(classes < s.vocab ? classes : s.vocab);
  const bool vec = aligned(L.from, 16) && aligned(L.to, 16) && (s.rows == 1 || s.ldy % 8 == 0) &&
                   (s.vocab == 1 || s.ldt % (L.grad_f32 ? 4 : 8) == 0);
  Chain chain{L.stream};
  return vec ? launch_scatter<true>(a, &chain) : launch_scatter<false>(a, &chain);
}

}  // namespace zeroadam
