// embedding.cu -- rows of a table looked up by token ids, and the gradient of the
// table, on sm_103a.
#include "chain.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "row_reads.hpp"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

__device__ __forceinline__ int64_t id_at(const void* ids, int32_t i32, int64_t i) {
  return i32 ? __ldg(static_cast<const int32_t*>(ids) + i)
             : __ldg(static_cast<const long long*>(ids) + i);
}

// 16 bytes, or zeros: a predicate and no branch, so that several are under way together
// (loads behind branches came one after the other: 4 us for 8 of them instead of 1).
__device__ __forceinline__ uint4 load16_if(bool p, const void* from) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n"
      " mov.b32 %3, 0;\n @p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(from), "r"(static_cast<int>(p)));
  return v;
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
        v[k] = load16_if(known && j + 8 <= a.width, from + j);
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
// keeping the rows' order, sums each token's rows in registers, and writes them; the rows
// of the table of no token are zeros, which a warp of its own gives to the TMA engine
// meanwhile.  Neither sums nor places go through atomics on floats or other blocks, so the
// result follows from the ids alone.
// Bound by the writes: 206 MB of zeros and sums at 8192 x 2048 of 50257.  (Clusters whose
// blocks look through a share of the ids each found their rows in half the time, but took
// 15 us longer from one call to the next.)

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kScatterThreads = kSumThreads + 32;  // and the warp of the zeros
constexpr int kSlice = 256;      // columns: 8 a lane
constexpr int kWindow = 4096;    // tokens of a class that are sorted at one time
constexpr int kMostRows = 6144;  // rows that are sorted at one time
constexpr int kEachRows = kMostRows / kSumWarps;  // of them, those that one warp finds
constexpr int kOneWarp = 48;     // rows of a token that one warp sums by itself

// The summing warps.
__device__ __forceinline__ void sum_sync() {
  asm volatile("barrier.sync.aligned 1, %0;" ::"n"(kSumThreads) : "memory");
}

struct ScatterArgs {
  const uint16_t* dy;
  const void* ids;
  void* dtable;
  int64_t rows, width, vocab, ldy, ldt, padding;
  int32_t ids_i32, grad_f32, accumulate;
  int32_t classes, slices;
  int32_t blocks;     // that share a token's rows (few tokens)
  WholeRows whole;    // rows of dy
  uint64_t inverse;   // 2^64 / classes, rounded up: its high product with an id is the quotient
  int32_t out_vec;    // rows of dtable are on 16 bytes
  int32_t bulk;       // a row of dtable is whole 16-byte vectors: zeros go by the TMA engine
  float scale;
};

constexpr int kZeros = 4096;  // bytes of zeros

struct ScatterShared {
  alignas(128) uint8_t zeros[kZeros];
  int32_t offset[kWindow + 1];  // counts; then where a token's rows begin; then where they end
  int32_t row[kMostRows];       // the class's rows in their order, kEachRows for each warp
  uint16_t token[kMostRows];    // and their tokens, within the window
  int32_t next;                 // share of the sums that is taken next
  int32_t full;                 // a warp has found more rows than there is room for
  int32_t sorted[kMostRows];    // rows by token
  uint16_t sorted_token[kMostRows];
  float part[kSumWarps][kSlice];
  int32_t found[kSumWarps];     // rows that each warp has found
  int32_t scan[kSumWarps];
  uint16_t common[kMostRows / kOneWarp];  // tokens of more than kOneWarp rows
  int32_t commons;
  uint32_t empty[kWindow / 32]; // tokens of no row, a bit each
};

// The 8 elements from the s-th on of a lane's aligned vector and the next lane's (lane 31's: `edge`);
// s is alike for the warp.
__device__ __forceinline__ uint4 from_column(uint4 v, uint4 edge, int s, int lane) {
  uint32_t w[8] = {v.x, v.y, v.z, v.w};
  const uint32_t e[4] = {edge.x, edge.y, edge.z, edge.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t next = __shfl_down_sync(0xffffffffu, w[k], 1);
    w[4 + k] = lane == 31 ? e[k] : next;
  }
  if (s & 4)
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  if (s & 2)
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  if (s & 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes that may lie in part outside dy, or zeros.
__device__ __forceinline__ uint4 vector_of(const Extents& in, bool has, uintptr_t p) {
  if (!has) return make_uint4(0, 0, 0, 0);
  if (in.whole(p)) return __ldg(reinterpret_cast<const uint4*>(p));
  uint64_t w[2];
  read_cut(p, in, w, [](uintptr_t q) { return __ldg(reinterpret_cast<const uint16_t*>(q)); });
  return make_uint4(static_cast<uint32_t>(w[0]), static_cast<uint32_t>(w[0] >> 32), static_cast<uint32_t>(w[1]),
                    static_cast<uint32_t>(w[1] >> 32));
}

// A lane's sums and 8 columns of a row whose vectors may lie in part outside dy.  (Not inlined: it
// would cost the loop beside it registers.)
struct Run {
  float x[8];
};
__device__ __noinline__ Run careful_row(const ScatterArgs& a, const uint16_t* row, int64_t n, int lane, Run run) {
  const uintptr_t begin = reinterpret_cast<uintptr_t>(a.dy), at = reinterpret_cast<uintptr_t>(row);
  const Extents in{begin, begin + 2 * ((a.rows - 1) * a.ldy + a.width)};
  const LaneReads r(at, n, lane);
  const uint4 low = vector_of(in, r.has_first, r.first), next = vector_of(in, r.has_next, r.next);
  float x[8];
  bf16x8(from_column(low, next, LaneReads::shift(at), lane), x);
#pragma unroll
  for (int c = 0; c < 8; ++c) run.x[c] += x[c];
  return run;
}

// How rows of dy lie.
enum Lie {
  kWhole,     // on 16 bytes, and whole vectors of them
  kAligned,   // on 16 bytes
  kAnywhere,
};

// The sum of a run of rows: 8 columns a lane, in the order of the rows, eight rows' loads
// under way at a time.  Rows that are not on 16 bytes come in aligned vectors too, shifted between
// lanes.  A lane's vector may end past the row, or begin before it: what is there goes into
// columns that no one writes.  Vectors that are not whole in dy's memory, of the first and last
// rows, are read element by element: a group of rows with one of these goes row by row (8192 x
// 2047 of 50257 83 us; with a look at each vector 99).  A chain ends after 64 rows, so that its
// error does not grow with a common token's count.
template <Lie LIE>
struct SliceSum {
  static constexpr bool VEC = LIE != kAnywhere, CUT = LIE != kWhole;
  float run[8] = {}, sum[8] = {};
  int chain = 0;

  // Rows rows[0], ..., rows[U - 1], those whose bit of `here` is set; after(u) follows the u-th.
  // careful (alike for the warp): some of them may not be whole.
  template <int U, typename After>
  __device__ __forceinline__ void walk(const ScatterArgs& a, const int32_t* rows, uint32_t here, int64_t col,
                                       int lane, bool careful, After after) {
    const uint16_t* const first = a.dy + col;
    const int64_t n = a.width - col;  // (lanes from there on have nothing)
    if (CUT && careful) {
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        if ((here >> u & 1) == 0) continue;
        Run now;
#pragma unroll
        for (int c = 0; c < 8; ++c) now.x[c] = run[c];
        now = careful_row(a, first + rows[u] * a.ldy, n, lane, now);
#pragma unroll
        for (int c = 0; c < 8; ++c) run[c] = now.x[c];
        after(u);
      }
      return;
    }
    uint4 v[U], edge[VEC ? 1 : U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool take = here >> u & 1;
      const uint16_t* from = first + (take ? rows[u] : 0) * a.ldy;
      if constexpr (VEC) {
        v[u] = load16_if(take && 8 * lane < n, from + 8 * lane);
      } else {
        // (as LaneReads has them)
        const int s = LaneReads::shift(reinterpret_cast<uintptr_t>(from));
        v[u] = load16_if(take && 8 * lane - s < n, from + 8 * lane - s);
        edge[u] = load16_if(take && lane == 31 && s > 0 && 256 - s < n, from + 256 - s);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((here >> u & 1) == 0) continue;
      if constexpr (!VEC)
        v[u] = from_column(v[u], edge[u], LaneReads::shift(reinterpret_cast<uintptr_t>(first + rows[u] * a.ldy)), lane);
      float x[8];
      bf16x8(v[u], x);
#pragma unroll
      for (int c = 0; c < 8; ++c) run[c] += x[c];
      after(u);
    }
  }
  // Rows in ascending order.  cut: there may be some among them that are not whole.
  __device__ __forceinline__ void add(const ScatterArgs& a, const int32_t* rows, int n, int64_t col,
                                      int lane, bool cut) {
    constexpr int U = 8;
#pragma unroll 1
    for (int k = 0; k < n; k += U) {
      const uint32_t here = n - k >= U ? (1u << U) - 1u : (1u << (n - k)) - 1u;
      const bool careful =
          CUT && cut && (rows[k] < a.whole.first || rows[n - k >= U ? k + U - 1 : n - 1] >= a.whole.end);
      walk<U>(a, rows + k, here, col, lane, careful, [](int) {});
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

__device__ __forceinline__ void add_vector(float* to, const float* x) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3])
               : "memory");
}

// A lane's 8 columns of one row of the table's gradient.
__device__ __forceinline__ void put_slice(const ScatterArgs& a, int64_t v, int64_t col, const float x[8],
                                          int lane) {
  const int64_t at = v * a.ldt + col;
  if (a.out_vec && col + 8 * lane + 8 <= a.width) {
    if (a.grad_f32) {
      float* o = static_cast<float*>(a.dtable) + at + 8 * lane;
      if (a.accumulate) {
        // One addition an element and call, in L2: nothing waits for what was there, and
        // there is no order to depend on.  (What comes to below 2^-126 is 0 there.)
        add_vector(o, x);
        add_vector(o + 4, x + 4);
      } else {
        reinterpret_cast<float4*>(o)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
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
    const int64_t j = 8 * lane + c;
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
  // an id's token within the window, or -1
  __device__ __forceinline__ int token_of(const ScatterArgs& a, int64_t id) const {
    const uint32_t k =
        classes == 1 ? static_cast<uint32_t>(id)
                     : static_cast<uint32_t>(__umul64hi(static_cast<uint32_t>(id), a.inverse));
    const int64_t t = static_cast<int64_t>(k) - w0;
    const bool good = id >= 0 && id < a.vocab && id != a.padding &&
                      static_cast<uint32_t>(id) - k * classes == mine && t >= 0 && t < window;
    return good ? static_cast<int>(t) : -1;
  }
};

// The sum of a token's rows, scaled and written.
template <Lie LIE>
__device__ __forceinline__ void finish_token(const ScatterArgs& a, const ScatterPlace& p, SliceSum<LIE>& s,
                                             int t, int lane) {
  s.join();
#pragma unroll
  for (int c = 0; c < 8; ++c) s.sum[c] *= a.scale;
  put_slice(a, (p.w0 + t) * p.classes + p.mine, p.col, s.sum, lane);
}

// n rows by the whole block: a run of them a warp, the warps' sums added in their order.
template <Lie LIE>
__device__ __forceinline__ void finish_token_together(const ScatterArgs& a, const ScatterPlace& p,
                                                      ScatterShared& sh, SliceSum<LIE>& s, int t) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  s.join();
#pragma unroll
  for (int c = 0; c < 8; ++c) sh.part[warp][32 * c + lane] = s.sum[c];
  sum_sync();
  if (warp == 0) {
    for (int k = 1; k < kSumWarps; ++k)
#pragma unroll
      for (int c = 0; c < 8; ++c) s.sum[c] += sh.part[k][32 * c + lane];
    finish_token(a, p, s, t, lane);
  }
  sum_sync();
}
template <Lie LIE>
__device__ __forceinline__ void add_share(const ScatterArgs& a, const ScatterPlace& p, SliceSum<LIE>& s,
                                          const int32_t* rows, int n) {
  const int warp = threadIdx.x / 32, per = (n + kSumWarps - 1) / kSumWarps;
  const int first = warp * per < n ? warp * per : n, end = first + per < n ? first + per : n;
  s.add(a, rows + first, end - first, p.col, threadIdx.x % 32, true);
}

// Rows [i0, i1) of tokens [t0, t1) in their order, each warp's own run of rows in its own
// part of the list (the first kEachRows of them); count: adds up offset[] too.  The list, found[]
// and full can be read after it.
__device__ __forceinline__ void list_rows(const ScatterArgs& a, const ScatterPlace& p, ScatterShared& sh, int64_t i0,
                                          int64_t i1, int t0, int t1, bool count) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t each = (i1 - i0 + kSumThreads - 1) / kSumThreads * 32;
  const int64_t from = i0 + warp * each, to = from + each < i1 ? from + each : i1;
  int n = 0;
  constexpr int U = 8;  // loads under way: what bounds this is their latency
  for (int64_t i = from; i < to; i += 32 * U) {
    int64_t id[U];  // (past the end: the last one, which does not count)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = i + 32 * u + lane;
      id[u] = id_at(a.ids, a.ids_i32, k < to ? k : to - 1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = i + 32 * u + lane;
      const int t = p.token_of(a, id[u]);
      const bool has = k < to && t >= t0 && t < t1;
      const uint32_t all = __ballot_sync(0xffffffffu, has);
      if (has) {
        const int at = n + __popc(all & ((1u << lane) - 1u));
        if (at < kEachRows) {
          sh.row[warp * kEachRows + at] = static_cast<int32_t>(k);
          sh.token[warp * kEachRows + at] = static_cast<uint16_t>(t);
        }
        if (count) atomicAdd(&sh.offset[t], 1);
      }
      n += __popc(all);
    }
  }
  if (lane == 0) {
    sh.found[warp] = n;
    if (n > kEachRows) sh.full = 1;
  }
  sum_sync();
}

// The listed rows by token, each token's in the order of the list: a warp takes every 8th
// token.  sorted[offset[t] - start ...], and offset[t] becomes the end.
__device__ __forceinline__ void sort_rows(ScatterShared& sh, int start) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int w = 0; w < kSumWarps; ++w) {
    const int n = sh.found[w];
    for (int k = w * kEachRows; k < w * kEachRows + n; k += 32) {
      const int t = k + lane < w * kEachRows + n ? sh.token[k + lane] : -1;
      const bool take = t >= 0 && t % kSumWarps == warp;
      const uint32_t takers = __ballot_sync(0xffffffffu, take);
      if (take) {
        const uint32_t same = __match_any_sync(takers, t);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int at = sh.offset[t];
        sh.sorted[at - start + before] = sh.row[k + lane];
        sh.sorted_token[at - start + before] = static_cast<uint16_t>(t);
        __syncwarp(takers);
        if (before == 0) sh.offset[t] = at + __popc(same);
      }
      __syncwarp();
    }
  }
  sum_sync();
}

// The tokens of the n sorted rows, one after the other: a warp takes the next 16 rows that no
// other has taken, of them the tokens whose first row is there, and has eight rows' loads
// under way at a time whatever tokens they are of.  Tokens of more than kOneWarp rows are
// left out.  (Which warp sums a token does not change its sum.)
template <Lie LIE>
__device__ __forceinline__ void sum_tokens(const ScatterArgs& a, const ScatterPlace& p, ScatterShared& sh, int start,
                                           int n, int t_first, int lane) {
  constexpr int U = 8, kTaken = 16;
  const auto begin_of = [&](int t) { return (t == t_first ? start : sh.offset[t - 1]) - start; };
  const auto end_of = [&](int t) { return sh.offset[t] - start; };
  const auto next_first = [&](int k) {  // the first row at or after k that is a token's first
    if (k >= n) return n;
    const int t = sh.sorted_token[k];
    return begin_of(t) == k ? k : end_of(t);
  };
  for (;;) {
    int share = 0;
    if (lane == 0) share = atomicAdd(&sh.next, 1);
    share = __shfl_sync(0xffffffffu, share, 0) * kTaken;
    if (share >= n) return;
    const int end = next_first(share + kTaken);
    SliceSum<LIE> s;
    for (int k = next_first(share); k < end;) {
      const int t = sh.sorted_token[k];
      if (end_of(t) - begin_of(t) > kOneWarp) {
        k = end_of(t);
        continue;
      }
      const int m = end - k < U ? end - k : U;
      int token = -1, after = -2;
      if (lane < m) {
        token = sh.sorted_token[k + lane];
        after = k + lane + 1 < n ? sh.sorted_token[k + lane + 1] : -2;
      }
      // rows that count, and those that end a token
      const bool counts = lane < m && end_of(token) - begin_of(token) <= kOneWarp;
      const uint32_t here = __ballot_sync(0xffffffffu, counts);
      const uint32_t last = __ballot_sync(0xffffffffu, counts && token != after);
      const bool careful =
          SliceSum<LIE>::CUT && __any_sync(0xffffffffu, counts && !a.whole.has(sh.sorted[k + lane]));
      s.template walk<U>(a, sh.sorted + k, here, p.col, lane, careful, [&](int u) {
        if ((last >> u & 1) == 0) return;
        finish_token(a, p, s, sh.sorted_token[k + u], lane);
        s = SliceSum<LIE>();
      });
      k += m;
    }
  }
}

// Rows of the table of no token: zeros, a token a lane (a warp's work).  A class's blocks share
// them out by rows, whole ones.
__device__ __forceinline__ void write_zeros(const ScatterArgs& a, const ScatterPlace& p, const ScatterShared& sh,
                                            int slice, int slices, int lane) {
  const int size = a.grad_f32 ? 4 : 2;
  const int64_t bytes = a.width * size;
  for (int t0 = slice; t0 < p.window; t0 += 32 * slices) {
    const int t = t0 + slices * lane;
    const bool none = t < p.window && (sh.empty[t / 32] >> (t % 32) & 1) != 0;
    char* row = static_cast<char*>(a.dtable) + ((p.w0 + t) * p.classes + p.mine) * a.ldt * size;
    if (a.bulk) {
      if (none) {
        for (int64_t b = 0; b < bytes; b += kZeros)
          bulk_store(row + b, sh.zeros, static_cast<uint32_t>(bytes - b < kZeros ? bytes - b : kZeros));
      }
      bulk_commit();
    } else {
      uint32_t left = __ballot_sync(0xffffffffu, none);
      while (left != 0) {
        const int u = __ffs(left) - 1;
        left &= left - 1;
        // up to a 16-byte boundary, vectors, and what is left
        char* o = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(row), u));
        const int64_t up = static_cast<int64_t>(-reinterpret_cast<uintptr_t>(o) & 15u);
        const int64_t head = up < bytes ? up : bytes, body = (bytes - head) / 16 * 16;
        if (2 * lane < head) *reinterpret_cast<uint16_t*>(o + 2 * lane) = 0;
        for (int64_t j = 16 * lane; j < body; j += 512) *reinterpret_cast<uint4*>(o + head + j) = make_uint4(0, 0, 0, 0);
        if (2 * lane < bytes - head - body) *reinterpret_cast<uint16_t*>(o + head + body + 2 * lane) = 0;
      }
    }
  }
}

template <Lie LIE>
__global__ void __launch_bounds__(kScatterThreads, 2)
    embedding_scatter_kernel(const __grid_constant__ ScatterArgs a) {
  extern __shared__ uint8_t raw[];
  ScatterShared& sh = *reinterpret_cast<ScatterShared*>(raw + ((128u - (smem_addr(raw) & 127u)) & 127u));
  if (a.bulk && threadIdx.x < kZeros / 16) {
    *reinterpret_cast<uint4*>(sh.zeros + 16 * threadIdx.x) = make_uint4(0, 0, 0, 0);
    fence_async_shared();
  }
  wait_for_predecessor();
  launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slices = a.slices, slice = static_cast<int>(blockIdx.x / static_cast<uint32_t>(a.classes));
  ScatterPlace p;
  p.col = static_cast<int64_t>(slice) * kSlice;
  p.mine = blockIdx.x % static_cast<uint32_t>(a.classes);
  p.classes = a.classes;
  const int64_t tokens = (a.vocab - p.mine + p.classes - 1) / p.classes;  // of this class

  for (p.w0 = 0; p.w0 < tokens; p.w0 += kWindow) {
    const int window = tokens - p.w0 < kWindow ? static_cast<int>(tokens - p.w0) : kWindow;
    p.window = window;
    for (int t = threadIdx.x; t <= window; t += kScatterThreads) sh.offset[t] = 0;
    if (threadIdx.x < kWindow / 32) sh.empty[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.full = 0;
    __syncthreads();
    if (warp == kSumWarps) {
      __syncthreads();  // the tokens of no row are known
      if (!a.accumulate) write_zeros(a, p, sh, slice, slices, lane);
      __syncthreads();  // the window is done
      continue;
    }
    list_rows(a, p, sh, 0, a.rows, 0, window, true);
    const bool room = sh.full == 0;
    // counts to offsets: a thread takes a run of tokens
    {
      const int per = (window + kSumThreads - 1) / kSumThreads;
      const int t0 = threadIdx.x * per < window ? threadIdx.x * per : window;
      const int t1 = t0 + per < window ? t0 + per : window;
      int rows = 0;
      for (int t = t0; t < t1; ++t) {
        const int n = sh.offset[t];
        rows += n;
        if (n == 0) atomicOr(&sh.empty[t / 32], 1u << (t % 32));
      }
      int x = rows;
#pragma unroll
      for (int k = 1; k < 32; k *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, x, k);
        if (lane >= k) x += u;
      }
      if (lane == 31) sh.scan[warp] = x;
      __syncthreads();  // (the zeros may begin)
      int before = x - rows;
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w)
        if (w < warp) before += sh.scan[w];
      for (int t = t0; t < t1; ++t) {
        const int n = sh.offset[t];
        sh.offset[t] = before;
        before += n;
      }
      if (threadIdx.x == kSumThreads - 1) sh.offset[window] = before;
      sum_sync();
    }
    // Tokens from t0 up to t1: all, if their rows have room; else as many as fit however
    // they lie, and a token of more rows than that alone, its rows in runs.  The ids are read
    // once more for each.
    for (int t0 = 0; t0 < window;) {
      const int start = sh.offset[t0];
      int t1 = window;
      if (!room) {
        int lo = t0 + 1, hi = window;  // the last t1 whose rows have room, or t0 + 1
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (sh.offset[mid] - start <= kEachRows) lo = mid;
          else hi = mid - 1;
        }
        t1 = lo;
      }
      const int count = sh.offset[t1] - start;
      sum_sync();  // (all have read what is set anew here)
      if (threadIdx.x == 0) sh.commons = sh.next = 0;
      sum_sync();
      if (!room && count > kEachRows) {
        SliceSum<LIE> s;
        for (int64_t i = 0; i < a.rows; i += kMostRows) {
          const int64_t end = i + kMostRows < a.rows ? i + kMostRows : a.rows;
          list_rows(a, p, sh, i, end, t0, t1, false);  // (a warp looks at kEachRows rows)
          s.add(a, sh.row + warp * kEachRows, sh.found[warp], p.col, lane, true);
          sum_sync();
        }
        finish_token_together(a, p, sh, s, t0);
      } else if (count > 0) {
        if (!room) list_rows(a, p, sh, 0, a.rows, t0, t1, false);
        sort_rows(sh, start);
        const auto begin_of = [&](int t) { return t == t0 ? start : sh.offset[t - 1]; };
        for (int t = t0 + static_cast<int>(threadIdx.x); t < t1; t += kSumThreads)
          if (sh.offset[t] - begin_of(t) > kOneWarp)
            sh.common[atomicAdd(&sh.commons, 1)] = static_cast<uint16_t>(t);
        sum_tokens<LIE>(a, p, sh, start, count, t0, lane);
        sum_sync();
        // tokens of many rows, by all warps (in any order: each is written by itself)
        for (int k = 0; k < sh.commons; ++k) {
          const int t = sh.common[k], first = begin_of(t);
          SliceSum<LIE> s;
          add_share(a, p, s, sh.sorted + first - start, sh.offset[t] - first);
          finish_token_together(a, p, sh, s, t);
        }
      }
      t0 = t1;
    }
    __syncthreads();
  }
  if (a.bulk) bulk_wait_all();
}

// Few tokens: a cluster of up to 8 blocks takes one token and one slice, its blocks a run of the
// rows each and their warps a run of those.  Nothing is sorted: a warp lists the rows of its run
// that are the token's, and adds them up 64 or more at a time.  The warps' sums are added in
// their order, and the blocks'.  What bounds it is the latency of the rows' loads (16384 x 2048 of
// 2 tokens: 18 us; by the kernel above, where a token's rows are one block's, 123).
constexpr int kFewWarps = 16, kFewThreads = 32 * kFewWarps, kFewCluster = 8;
constexpr int kFewItems = 2 * kSms, kManyRows = 4096;
constexpr int kFewListed = 64, kFewAsked = 4;  // rows that are added up; loads of 32 ids under way

template <Lie LIE>
__global__ void __launch_bounds__(kFewThreads, 1)
    embedding_few_tokens_kernel(const __grid_constant__ ScatterArgs a) {
  __shared__ alignas(16) float part[kFewWarps][kSlice];
  __shared__ alignas(16) float sum[kSlice];
  __shared__ int32_t list[kFewWarps][kFewListed + 32 * kFewAsked];
  __shared__ int32_t found[kFewWarps], all;
  wait_for_predecessor();
  launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, blocks = a.blocks;
  const int rank = static_cast<int>(blockIdx.x) % blocks, item = static_cast<int>(blockIdx.x) / blocks;
  const int64_t token = item % a.vocab, col = static_cast<int64_t>(item / static_cast<int>(a.vocab)) * kSlice;
  const int64_t run = rank * kFewWarps + warp, runs = static_cast<int64_t>(blocks) * kFewWarps;
  const int64_t from = a.rows * run / runs, to = a.rows * (run + 1) / runs;
  const bool cut = from < a.whole.first || to > a.whole.end;
  SliceSum<LIE> s;
  int n = 0, rows = 0;
  for (int64_t i = from; token != a.padding && i < to; i += 32 * kFewAsked) {
    int64_t id[kFewAsked];
#pragma unroll
    for (int u = 0; u < kFewAsked; ++u) {
      const int64_t k = i + 32 * u + lane;
      id[u] = id_at(a.ids, a.ids_i32, k < to ? k : to - 1);
    }
#pragma unroll
    for (int u = 0; u < kFewAsked; ++u) {
      const int64_t k = i + 32 * u + lane;
      const bool has = k < to && id[u] == token;
      const uint32_t those = __ballot_sync(0xffffffffu, has);
      if (has) list[warp][n + __popc(those & ((1u << lane) - 1u))] = static_cast<int32_t>(k);
      n += __popc(those);
    }
    if (n < kFewListed && i + 32 * kFewAsked < to) continue;
    __syncwarp();
    s.add(a, list[warp], n, col, lane, cut);
    __syncwarp();
    rows += n;
    n = 0;
  }
  s.join();
  *reinterpret_cast<float4*>(&part[warp][8 * lane]) = make_float4(s.sum[0], s.sum[1], s.sum[2], s.sum[3]);
  *reinterpret_cast<float4*>(&part[warp][8 * lane + 4]) = make_float4(s.sum[4], s.sum[5], s.sum[6], s.sum[7]);
  if (lane == 0) found[warp] = rows;
  __syncthreads();
  if (threadIdx.x < kSlice) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) x += part[w][threadIdx.x];
    sum[threadIdx.x] = x;
  }
  if (threadIdx.x == 0) {
    int x = 0;
    for (int w = 0; w < kFewWarps; ++w) x += found[w];
    all = x;
  }
  if (blocks > 1) cluster_sync_writes();
  else __syncthreads();
  if (rank == 0 && warp == 0) {
    float x[8] = {};
    uint32_t any = 0;
    for (int r = 0; r < blocks; ++r) {
      const float4 lo = peer_load(peer_addr(&sum[8 * lane], r)), hi = peer_load(peer_addr(&sum[8 * lane + 4], r));
      x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
      x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
      any |= peer_load_u32(peer_addr(&all, r));
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] *= a.scale;
    if (any != 0 || !a.accumulate) put_slice(a, token, col, x, lane);  // (of no rows: 0, or as it was)
  }
  if (blocks > 1) cluster_sync();  // no block ends while another reads from it
}

template <Lie LIE>
cudaError_t launch_scatter(const ScatterArgs& a, Chain* chain) {
  constexpr int smem = static_cast<int>(sizeof(ScatterShared)) + 128;
  static_assert(smem <= 113 * 1024, "two blocks an SM");
  const auto kernel = embedding_scatter_kernel<LIE>;
  const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = int64_t{a.classes} * a.slices;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return chain->launch(kernel, dim3(static_cast<unsigned>(blocks)), kScatterThreads, smem, 1, a);
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
  const bool vec = aligned(L.from, 16) && (s.rows == 1 || s.ldy % 8 == 0);
  ScatterArgs a{};
  a.whole = WholeRows(s.rows, s.width, s.ldy, vec);
  const Lie lie = !vec ? kAnywhere : a.whole.end < s.rows ? kAligned : kWhole;
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
  const int64_t slices = (s.width + kSlice - 1) / kSlice;
  a.out_vec = aligned(L.to, 16) && (s.vocab == 1 || s.ldt % (L.grad_f32 ? 4 : 8) == 0);
  Chain chain{L.stream};
  // Few tokens: up to two blocks an SM with their slices, four where there are many rows (300 tokens
  // of 256 columns, 600 rows 5.4 us, by the other kernel 9.1; 600 tokens 9.2 and 8.1, but with
  // 8192 rows 15 and 23).  Clusters as large as the SMs have room for, and as leave every block 256
  // rows.
  if (s.vocab * slices <= (s.rows < kManyRows ? 1 : 2) * kFewItems) {
    a.blocks = 1;
    while (a.blocks < kFewCluster && 2 * a.blocks * s.vocab * slices <= kSms && s.rows >= 512 * a.blocks) a.blocks *= 2;
    return chain.launch(lie == kWhole     ? embedding_few_tokens_kernel<kWhole>
                        : lie == kAligned ? embedding_few_tokens_kernel<kAligned>
                                          : embedding_few_tokens_kernel<kAnywhere>,
                        dim3(static_cast<unsigned>(a.blocks * s.vocab * slices)), kFewThreads, 0, a.blocks, a);
  }
  // Two blocks an SM in all; more where a class would have over half of the rows that a block
  // has room for.
  a.slices = static_cast<int32_t>(slices);
  int64_t classes = 2 * kSms / slices;
  const int64_t least = s.rows / (kMostRows / 2) + 1;
  if (classes < least) classes = least;
  a.classes = static_cast<int32_t>(classes < s.vocab ? classes : s.vocab);
  a.inverse = a.classes > 1 ? ~uint64_t{0} / static_cast<uint64_t>(a.classes) + 1 : 0;
  a.bulk = a.out_vec && s.width * (L.grad_f32 ? 4 : 2) % 16 == 0;
  return lie == kWhole     ? launch_scatter<kWhole>(a, &chain)
         : lie == kAligned ? launch_scatter<kAligned>(a, &chain)
                           : launch_scatter<kAnywhere>(a, &chain);
}

}  // namespace zeroadam
