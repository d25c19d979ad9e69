// block_norm.cu -- the norms before and after a model's block with its gate and
// residual scale, forward and backward, on sm_103a:
//   s = r + alpha * gate * P(h),   y = N(s),
// a row at a time, in registers between its loads and its stores, so that each matrix is
// read or written once.  Bound by HBM: 8 bytes an element forward, 12 backward.
#include <type_traits>

#include "chain.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

constexpr int kMostThreads = 512, kMostWarps = kMostThreads / 32, kMostCluster = 8;
// Rows under way.  More of them make the forward pass slower where HBM bounds it (32768 x 2048 with
// 2, 3, 4: 83, 96, 98 us), fewer the backward pass (2, 3, 4 without a norm after the block: 119, 110,
// 85 us).
constexpr int kForwardStages = 2, kBackwardStages = 4;
constexpr int kSumsAtOnce = 8;

// Who shares a row: a block up to 4,096 columns, a cluster of blocks beyond.  A thread has 8
// columns in every case, so that the backward pass has room for the sums of each in
// registers, and the vectors are read once.
enum Share { kBlock, kCluster };

__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// What a row is read from.
// (the backward pass's s is kInR; it always has that and kInDy, the forward kInR)
enum Input { kInDy, kInR, kInDs, kInH, kInGate, kInputs };

struct NormArgs {
  int64_t rows, width;
  int32_t post, kind;
  float alpha, eps;
  const uint16_t* in[kInputs];  // NULL: not there (kInR is the backward pass's s)
  uint32_t pitch[kInputs];      // bytes
  int32_t inputs;               // how many are there
  const uint16_t *gate, *w1, *b1, *w, *b;  // vectors (gate: or NULL, kInGate is a matrix)
  uint16_t *s_out, *y;
  uint16_t *dr, *dh, *dgate_rows;          // dgate_rows: a matrix
  uint32_t pitch_s, pitch_y, pitch_dr, pitch_dh, pitch_dg;  // bytes
  int32_t wvec;    // the vectors are read 16 bytes at a time
  // backward: sums of each block's rows, [kSums][blocks][width], where wanted
  float* sums;
  int32_t blocks;
  int32_t wanted;  // bit q: sum q
};

// The sums over rows.
enum { kDw, kDgate, kDw1, kDb, kDb1, kSums };

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t from) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(from)
               : "memory");
  return v;
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's 8 columns of a row, in fp32, two to an operation: with one at a time the kernels
// were bound by their instructions (500 a row and warp forward, 780 backward).
struct Eight {
  Pair p[4];
};
__device__ __forceinline__ Eight all_of(float x) {
  Eight r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.p[k] = pair(x, x);
  return r;
}
__device__ __forceinline__ Eight eight_of(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Eight r;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    r.p[k] = pair(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  return r;
}
__device__ __forceinline__ uint4 bf16_of(const Eight& x) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo, hi;
    split(x.p[k], lo, hi);
    w[k] = bf16x2_bits(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Eight operator*(const Eight& a, const Eight& b) {
  Eight r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.p[k] = a.p[k] * b.p[k];
  return r;
}
__device__ __forceinline__ Eight operator*(const Eight& a, float b) { return a * all_of(b); }
__device__ __forceinline__ Eight operator+(const Eight& a, const Eight& b) {
  Eight r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.p[k] = a.p[k] + b.p[k];
  return r;
}
__device__ __forceinline__ Eight fma8(const Eight& a, const Eight& b, const Eight& c) {
  Eight r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.p[k] = fma2(a.p[k], b.p[k], c.p[k]);
  return r;
}
__device__ __forceinline__ float total(Pair a, Pair b, Pair c, Pair d) {
  float lo, hi;
  split((a + b) + (c + d), lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float sum8(const Eight& a) { return total(a.p[0], a.p[1], a.p[2], a.p[3]); }
__device__ __forceinline__ float dot8(const Eight& a, const Eight& b) {
  float lo, hi;
  split(fma2(a.p[0], b.p[0], a.p[1] * b.p[1]) + fma2(a.p[2], b.p[2], a.p[3] * b.p[3]), lo, hi);
  return lo + hi;
}

// A thread's columns: a 16-byte vector (VEC), or 8 single ones spread over the row.
template <bool VEC>
struct Columns {
  int at, lanes, width;
  bool whole;  // all 8 are the row's, and may go as a vector
  __device__ __forceinline__ Columns(int at, int lanes, int width)
      : at(at), lanes(lanes), width(width), whole(VEC && 8 * at + 8 <= width) {}
  __device__ __forceinline__ int of(int k) const { return VEC ? 8 * at + k : k * lanes + at; }
  __device__ __forceinline__ bool in(int k) const { return of(k) < width; }
  // Elements one by one (0 past the row's end).
  __device__ __forceinline__ Eight load_single(const uint16_t* p) const {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = in(k) ? bf16_at(p + of(k)) : 0.0f;
    Eight r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.p[k] = pair(x[2 * k], x[2 * k + 1]);
    return r;
  }
  // A vector of the columns (NULL: `other`), which lies on 16 bytes or not.
  __device__ __forceinline__ Eight load_vector(const uint16_t* p, float other, bool vec) const {
    if (p == nullptr) return all_of(other);
    if (vec && whole) return eight_of(__ldg(reinterpret_cast<const uint4*>(p + 8 * at)));
    return load_single(p);
  }
  __device__ __forceinline__ void store(uint16_t* p, const Eight& x) const {
    if (whole) {
      *reinterpret_cast<uint4*>(p + 8 * at) = bf16_of(x);
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      split(x.p[k], lo, hi);
      if (in(2 * k)) p[of(2 * k)] = to_bf16(lo);
      if (in(2 * k + 1)) p[of(2 * k + 1)] = to_bf16(hi);
    }
  }
  // Columns past the row's end set to 0 (a thread that has some).
  __device__ __forceinline__ void clear(Eight& x) const {
    if (whole) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      split(x.p[k], lo, hi);
      x.p[k] = pair(in(2 * k) ? lo : 0.0f, in(2 * k + 1) ? hi : 0.0f);
    }
  }
};

// A vector of the columns in bf16, 4 registers instead of 8 (NULL: ones).
struct Held {
  uint4 v;
  template <bool VEC>
  __device__ __forceinline__ Held(const Columns<VEC>& at, const uint16_t* p, bool vec)
      : v(bf16_of(at.load_vector(p, 1.0f, vec))) {}
  __device__ __forceinline__ Eight get() const { return eight_of(v); }
};

// Values that stay in registers: without this the compiler works out flags, pitches and places
// anew from the kernel's arguments for every row, 150 instructions of it.
__device__ __forceinline__ void keep(uint32_t& x) { asm volatile("" : "+r"(x)); }
__device__ __forceinline__ void keep(const uint16_t*& p) { asm volatile("" : "+l"(p)); }

// Row i of a matrix, from its first row's place for this thread.
__device__ __forceinline__ const uint16_t* row_at(const uint16_t* base, uint32_t i, uint32_t pitch) {
  return reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) +
                                           static_cast<uint64_t>(i) * pitch);
}

// The rows that a thread reads, STAGES under way (VEC): its own 16 bytes of each input, from its
// own place in shared memory, so no thread waits for another's.  Rows that are not on 16-byte
// boundaries are read when they are wanted.  FIRST to LAST: the inputs there may be.
template <bool VEC, int FIRST, int LAST, int STAGES>
struct Rows {
  const NormArgs& a;
  const Columns<VEC>& at;
  const uint16_t* base[kInputs];
  uint32_t there;                 // bit q: input q
  uint32_t place;                 // of the first input, in the first stage
  uint32_t stage, end;            // bytes of a stage, and of all
  uint32_t each;                  // bytes of an input in a stage
  uint32_t put = 0, got = 0;      // the stage asked into, and that read
  uint32_t next, step, rows;

  __device__ __forceinline__ Rows(const NormArgs& a, const Columns<VEC>& at, uint8_t* ring, uint32_t first,
                                  uint32_t step)
      : a(a), at(at), there(0), each(blockDim.x * 16), next(first), step(step),
        rows(static_cast<uint32_t>(a.rows)) {
    place = smem_addr(ring) + threadIdx.x * 16;
    stage = a.inputs * each;
    end = STAGES * stage;
#pragma unroll
    for (int q = FIRST; q <= LAST; ++q) {
      there |= (a.in[q] != nullptr ? 1u : 0u) << q;
      base[q] = a.in[q] + (VEC ? 8 * at.at : 0);
      keep(base[q]);
    }
    keep(there);
    keep(stage);
    keep(end);
    keep(each);
  }
  __device__ __forceinline__ bool has(int q) const { return (there >> q & 1u) != 0; }
  __device__ __forceinline__ void ask() {
    if (next < rows && at.whole) {
      uint32_t to = place + put;  // the inputs that are there, one after the other
#pragma unroll
      for (int q = FIRST; q <= LAST; ++q)
        if (has(q)) {
          copy16(to, row_at(base[q], next, a.pitch[q]));
          to += each;
        }
    }
    next += step;
    put = put + stage == end ? 0 : put + stage;
    copy_commit();
  }
  __device__ __forceinline__ void begin() {
    if constexpr (VEC) {
#pragma unroll
      for (int k = 1; k < STAGES; ++k) ask();
    }
  }
  // The next R rows can be read.
  __device__ __forceinline__ void arrive(int R = 1) {
    if constexpr (VEC) {
      ask();
      if (R > 1) {
        copy_wait<STAGES - 2>();  // (all but the last two)
      } else {
        copy_wait<STAGES - 1>();
      }
    }
  }
  // Input q of row i, that is the `nth` of the inputs that are there, `ahead` of the rows read.
  __device__ __forceinline__ Eight read(int q, uint32_t i, uint32_t nth, int ahead = 0) const {
    if constexpr (VEC) {
      uint32_t from = got;
      if (ahead > 0) from = from + stage == end ? 0 : from + stage;
      if (at.whole) return eight_of(shared16(place + from + nth * each));
      return at.load_single(row_at(base[q] - 8 * at.at, i, a.pitch[q]));
    } else {
      return at.load_single(row_at(base[q], i, a.pitch[q]));
    }
  }
  // R rows have been read (another may be asked for in the place of each but the last).
  __device__ __forceinline__ void done(int R = 1) {
    if constexpr (VEC) {
      got = got + stage == end ? 0 : got + stage;
      if (R > 1) {
        ask();
        got = got + stage == end ? 0 : got + stage;
      }
    }
  }
};

// A matrix that is written by rows.
template <bool VEC>
struct Output {
  const uint16_t* base;
  uint32_t pitch;
  __device__ __forceinline__ Output(uint16_t* p, uint32_t pitch) : base(p), pitch(pitch) { keep(base); }
  __device__ __forceinline__ void put(const Columns<VEC>& at, uint32_t i, const Eight& x) const {
    if (base != nullptr) at.store(const_cast<uint16_t*>(row_at(base, i, pitch)), x);
  }
};

// N sums over the threads of a row (or of two), alike for each of them.  A warp adds up its
// lanes' by halves: where there are several sums, each step passes on half of them, so 4 sums
// take 6 exchanges and not 20.  The warps' parts go through shared memory, every block's to all
// blocks of the cluster, in two places taken in turn, so that one barrier is enough: a
// place is written again only after the barrier that follows its reading.
template <Share SHARE>
struct RowSum {
  static constexpr int kParts = SHARE == kBlock ? 32 : kMostCluster * kMostWarps;
  float (*part)[kParts][kSumsAtOnce];  // kBlock: parts past the block's warps are 0
  int place = 0;
  __device__ __forceinline__ static float from(float x, int k) { return __shfl_xor_sync(0xffffffffu, x, k); }
  // The sum of x[lane % N] over the lanes (N 1, 2, 4 or 8).
  template <int N>
  __device__ __forceinline__ static float over_lanes(const float (&x)[N], int lane) {
    float v;
    if constexpr (N == 1) {
      v = x[0] + from(x[0], 1);
      v += from(v, 2);
    } else if constexpr (N == 2) {
      const bool odd = lane & 1;
      v = (odd ? x[1] : x[0]) + from(odd ? x[0] : x[1], 1);
      v += from(v, 2);
    } else {
      const bool odd = lane & 1, high = lane & 2;
      float y[N / 4];
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const float* z = x + 4 * k;
        const float lo = (odd ? z[1] : z[0]) + from(odd ? z[0] : z[1], 1);
        const float hi = (odd ? z[3] : z[2]) + from(odd ? z[2] : z[3], 1);
        y[k] = (high ? hi : lo) + from(high ? lo : hi, 2);
      }
      v = y[0];
      if constexpr (N == 8) {
        const bool top = lane & 4;
        v = (top ? y[1] : y[0]) + from(top ? y[0] : y[1], 4);
      }
    }
    if constexpr (N != 8) v += from(v, 4);
    v += from(v, 8);
    v += from(v, 16);
    return v;
  }
  template <int N>
  __device__ __forceinline__ void operator()(float (&x)[N]) {
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int W = N == 8 ? 8 : 4;  // of a part, N of them in use; lane l takes sum l % W of
                                       // the parts l / W, l / W + 32 / W, ...
    float v = over_lanes(x, lane);
    if (SHARE == kCluster || warps > 1) {
      int parts = kMostWarps;
      if constexpr (SHARE == kBlock) {
        if (lane < W) part[place][warp][lane] = v;
        __syncthreads();
      } else {
        const int blocks = static_cast<int>(cluster_blocks());
        for (int k = lane; k < W * blocks; k += 32)  // to block k / W (the lanes' sums repeat every W)
          peer_store(peer_addr(&part[place][static_cast<int>(cluster_rank()) * warps + warp][k % W], k / W), v);
        __syncwarp();
        cluster_sync_writes();
        parts = blocks * warps;
      }
      v = 0.0f;
      if constexpr (SHARE == kBlock) {
#pragma unroll
        for (int w = 0; w < kMostWarps; w += 32 / W)
          if (w < warps) v += part[place][lane / W + w][lane % W];
      } else {
        for (int w = lane / W; w < parts; w += 32 / W) v += part[place][w][lane % W];
        __syncwarp();
      }
      if constexpr (W == 4) v += from(v, 4);
      v += from(v, 8);
      v += from(v, 16);
      place ^= 1;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = __shfl_sync(0xffffffffu, v, n);
  }
};

// A row's threads, and which rows they take.
template <Share SHARE>
struct RowOwner {
  int at, lanes;        // this thread's place among the row's
  uint32_t first, step;  // rows
  __device__ __forceinline__ RowOwner() {
    const int blocks = SHARE == kBlock ? 1 : static_cast<int>(cluster_blocks());
    at = SHARE == kBlock ? threadIdx.x : cluster_rank() * blockDim.x + threadIdx.x;
    lanes = blocks * blockDim.x;
    first = blockIdx.x / blocks;
    step = gridDim.x / blocks;
  }
};

// Before the first sum: a block's parts that no warp writes are 0; a cluster's blocks are there.  (A
// cluster's parts are all written, by other blocks too: a 0 put here could come after those.)
template <Share SHARE>
__device__ __forceinline__ void begin_sums(float (*part)[RowSum<SHARE>::kParts][kSumsAtOnce]) {
  if constexpr (SHARE == kCluster) {
    cluster_sync();
  } else {
    for (int k = threadIdx.x; k < 2 * RowSum<SHARE>::kParts * kSumsAtOnce; k += blockDim.x)
      (&part[0][0][0])[k] = 0.0f;
    __syncthreads();
  }
}

// What norms there are, in one register.  LAYER: there may be norms of that kind.
template <bool LAYER>
struct Kinds {
  uint32_t bits;
  __device__ __forceinline__ explicit Kinds(const NormArgs& a)
      : bits((a.kind == ZERO_NORM_LAYER ? 1u : 0u) | (a.post == ZERO_NORM_LAYER ? 2u : 0u) |
             (a.post != ZERO_NORM_NONE ? 4u : 0u)) {
    keep(bits);
  }
  __device__ __forceinline__ bool layer() const { return LAYER && (bits & 1u) != 0; }
  __device__ __forceinline__ bool post_layer() const { return LAYER && (bits & 2u) != 0; }
  __device__ __forceinline__ bool post() const { return (bits & 4u) != 0; }
};

// LAYER: there are norms of that kind, or biases, which are theirs.
template <bool VEC, Share SHARE, bool LAYER>
__global__ void __launch_bounds__(kMostThreads, 2)
    block_norm_forward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][RowSum<SHARE>::kParts][kSumsAtOnce];
  extern __shared__ uint8_t ring[];
  wait_for_predecessor();
  launch_dependents();
  const RowOwner<SHARE> own;
  const Columns<VEC> at(own.at, own.lanes, static_cast<int>(a.width));
  Rows<VEC, kInR, kInGate, kForwardStages> rows(a, at, ring, own.first, own.step);
  rows.begin();
  const Output<VEC> s_out(a.s_out, a.pitch_s), y_out(a.y, a.pitch_y);
  const bool wvec = a.wvec != 0;
  const Kinds<LAYER> kinds(a);
  // s = r + (h standardized * scale1 + bias1) [* gate's row]
  Eight scale1 = at.load_vector(a.gate, 1.0f, wvec) * a.alpha, bias1 = all_of(0.0f);
  if constexpr (LAYER) bias1 = at.load_vector(a.b1, 0.0f, wvec) * scale1;
  scale1 = scale1 * at.load_vector(a.w1, 1.0f, wvec);
  const Eight w = at.load_vector(a.w, 1.0f, wvec), b = LAYER ? at.load_vector(a.b, 0.0f, wvec) : all_of(0.0f);
  begin_sums<SHARE>(part);
  RowSum<SHARE> row_sum{part};
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const bool layer = kinds.layer(), post_layer = kinds.post_layer();
  const auto center = [&](Eight& x, float sum) {
    x = x + all_of(-sum * inv_width);
    at.clear(x);
  };
  const auto inverse_of = [&](float squares) { return rsqrtf(fmaf(squares, inv_width, a.eps)); };
  // s of row i, from r and h standardized
  const auto add = [&](uint32_t i, Eight s, const Eight& h) {
    if (rows.has(kInGate)) {
      Eight p = h * scale1;
      if constexpr (LAYER) p = p + bias1;
      s = fma8(p, rows.read(kInGate, i, 2), s);
    } else {
      if constexpr (LAYER) s = s + bias1;
      s = fma8(h, scale1, s);
    }
    s_out.put(at, i, s);
    if constexpr (LAYER)
      if (layer) at.clear(s);
    return s;
  };
  const auto end = [&](uint32_t i, Eight& s, float squares) {
    s = s * inverse_of(squares);
    if constexpr (LAYER) s = fma8(s, w, b);
    else s = s * w;
    y_out.put(at, i, s);
  };
  if (VEC && kinds.post()) {
    // The sums of a row's s are taken with those of the next row's h: one wait a row, not two
    // (8192 x 2048 26 -> 23 us, 4096 x 8192 in clusters 93 -> 66).  Rows that are not asked for ahead
    // are better one by one, r beside h (1003 x 775 9 us, in turn 15).
    Eight s = all_of(0.0f);
    for (uint32_t i = own.first;; i += own.step) {
      const bool more = i < rows.rows, before = i != own.first;
      if (!more && !before) break;
      Eight h = all_of(0.0f);
      if (more) {
        rows.arrive();
        h = rows.read(kInH, i, 1);
      }
      if (layer || post_layer) {
        float m[2] = {sum8(h), sum8(s)};
        row_sum(m);
        if (post_layer) center(h, m[0]);
        if (layer) center(s, m[1]);
      }
      float q[2] = {dot8(h, h), dot8(s, s)};
      row_sum(q);
      if (before) end(i - own.step, s, q[1]);
      if (!more) break;
      s = add(i, rows.read(kInR, i, 0), h * inverse_of(q[0]));
      rows.done();
    }
  } else {
    for (uint32_t i = own.first; i < rows.rows; i += own.step, rows.done()) {
      rows.arrive();
      Eight s = rows.read(kInR, i, 0);
      if (rows.has(kInH)) {
        Eight h = rows.read(kInH, i, 1);
        if (!VEC && kinds.post()) {
          if (post_layer) {
            float m[1] = {sum8(h)};
            row_sum(m);
            center(h, m[0]);
          }
          float q[1] = {dot8(h, h)};
          row_sum(q);
          h = h * inverse_of(q[0]);
        }
        s = add(i, s, h);
      } else {
        s_out.put(at, i, s);
      }
      if (layer) {
        float m[1] = {sum8(s)};
        row_sum(m);
        center(s, m[0]);
      }
      float q[1] = {dot8(s, s)};
      row_sum(q);
      end(i, s, q[0]);
    }
  }
  if constexpr (SHARE == kCluster) cluster_sync();  // no block ends while others write to it
}

// The backward pass: a block (or cluster) takes every so-many-th row, its threads the same 8
// columns of each, whose sums over the rows stay in their registers until the end.  With xh
// the standardized row, u what reaches it and m its means,
//   x's gradient = (u - m(u) [LAYER] - xh m(u xh)) / root.
// FULL: there is a norm after the block, or a gate: h is read.
template <bool VEC, Share SHARE, bool FULL, bool LAYER>
__global__ void __launch_bounds__(kMostThreads)
    block_norm_backward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][RowSum<SHARE>::kParts][kSumsAtOnce];
  extern __shared__ uint8_t ring[];
  wait_for_predecessor();
  launch_dependents();
  const RowOwner<SHARE> own;
  const Columns<VEC> at(own.at, own.lanes, static_cast<int>(a.width));
  Rows<VEC, kInDy, kInGate, kBackwardStages> rows(a, at, ring, own.first, own.step);
  rows.begin();
  const Output<VEC> dr_out(a.dr, a.pitch_dr), dh_out(a.dh, a.pitch_dh), dgate_out(a.dgate_rows, a.pitch_dg);
  const bool wvec = a.wvec != 0;
  const Kinds<LAYER> kinds(a);
  // With a = s's gradient (times the gate's row, where it is a matrix) and hh the standardized h,
  // what reaches hh is a c, c = alpha w1 (times the gate, where it is a vector), and the sums of
  // a hh and a over the rows give dw1, db1 and a vector's dgate.
  const Eight w = at.load_vector(a.w, 1.0f, wvec);
  const Held w1(at, FULL ? a.w1 : nullptr, wvec);  // (of a matrix gate's gradient alone)
  Eight c = all_of(a.alpha);
  if constexpr (FULL) c = (at.load_vector(a.gate, 1.0f, wvec) * a.alpha) * w1.get();
  Eight dw = all_of(0.0f), db = dw, ah = dw, aa = dw;
  begin_sums<SHARE>(part);
  RowSum<SHARE> row_sum{part};
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const bool layer = kinds.layer(), post_layer = kinds.post_layer(), post = kinds.post();
  const uint32_t has_ds = rows.has(kInDs) ? 1u : 0u;
  // What is done with a row i, `ahead` of the rows read, between its sums.  First means are taken off:
  const auto center = [&](Eight& x, Eight& h, const float* m) {
    if (layer) {
      x = x + all_of(-m[0] * inv_width);
      at.clear(x);
    }
    if constexpr (FULL)
      if (post_layer) {
        h = h + all_of(-m[1] * inv_width);
        at.clear(h);
      }
  };
  // then x x, u w x, h h, u w [LAYER]
  constexpr int Q = LAYER ? 4 : FULL ? 3 : 2, M = LAYER ? 2 : 1;
  const auto products = [&](const Eight& x, const Eight& u, const Eight& h, float* q) {
    const Eight uw = u * w;
    q[0] = dot8(x, x);
    q[1] = dot8(uw, x);
    if constexpr (Q > 2) q[2] = FULL ? dot8(h, h) : 0.0f;
    if constexpr (LAYER) q[3] = layer ? sum8(uw) : 0.0f;
  };
  // then dr; x becomes what reaches h's norm, h standardized, m their sums; h's 1 / root
  const auto through = [&](uint32_t i, int ahead, Eight& x, const Eight& u, Eight& h, const float* q, float* m) {
    const float inverse = rsqrtf(fmaf(q[0], inv_width, a.eps));
    const float along = q[1] * inverse * inv_width;
    float inverse1 = 1.0f;
    x = x * inverse;  // standardized
    dw = fma8(u, x, dw);
    if constexpr (LAYER) db = db + u;
    x = fma8(x, all_of(-along), u * w);
    if constexpr (LAYER)
      if (layer) x = x + all_of(-q[3] * inv_width);
    if (has_ds) x = fma8(x, all_of(inverse), rows.read(kInDs, i, 2, ahead));
    else x = x * inverse;
    if constexpr (LAYER) at.clear(x);  // (else they are 0 already)
    dr_out.put(at, i, x);
    if constexpr (FULL) {
      if (post) inverse1 = rsqrtf(fmaf(q[2], inv_width, a.eps));
      h = h * inverse1;
      if (rows.has(kInGate)) {
        Eight t = h * w1.get();
        if constexpr (LAYER) t = t + at.load_vector(a.b1, 0.0f, wvec);
        dgate_out.put(at, i, (x * a.alpha) * t);
        x = x * rows.read(kInGate, i, 3 + has_ds, ahead);
      }
      ah = fma8(x, h, ah);
      if constexpr (LAYER) aa = aa + x;
    }
    x = x * c;
    if constexpr (FULL) {
      m[0] = dot8(x, h);
      if constexpr (LAYER) m[1] = post_layer ? sum8(x) : 0.0f;
    }
    return inverse1;
  };
  // and dh.
  const auto end = [&](uint32_t i, Eight& x, const Eight& h, const float* m, float inverse1) {
    if (FULL && post) {
      x = fma8(h, all_of(-m[0] * inv_width), x);
      if constexpr (LAYER)
        if (post_layer) x = x + all_of(-m[1] * inv_width);
      x = x * inverse1;
    }
    dh_out.put(at, i, x);
  };
  // R rows, i and i + step: what they wait for, they wait for together.
  const auto make = [&](auto how_many, uint32_t i0) {
    constexpr int R = decltype(how_many)::value, QR = Q == 3 ? 4 : Q;
    Eight x[R], u[R], h[R];
    float q[QR * R] = {}, m[2 * R], inverse1[R];
    const auto each = [&](auto f) {
#pragma unroll
      for (int r = 0; r < R; ++r) f(r, i0 + r * own.step);
    };
    if constexpr (VEC) rows.arrive(R);
    each([&](int r, uint32_t i) {
      x[r] = rows.read(kInR, i, 1, r);
      u[r] = rows.read(kInDy, i, 0, r);
      if constexpr (FULL) h[r] = rows.read(kInH, i, 2 + has_ds, r);
    });
    if (layer || (FULL && post_layer)) {
      each([&](int r, uint32_t) {
        m[2 * r] = sum8(x[r]);
        m[2 * r + 1] = FULL ? sum8(h[r]) : 0.0f;
      });
      row_sum(m);
      each([&](int r, uint32_t) { center(x[r], h[r], m + 2 * r); });
    }
    each([&](int r, uint32_t) { products(x[r], u[r], h[r], q + QR * r); });
    row_sum(q);
    each([&](int r, uint32_t i) { inverse1[r] = through(i, r, x[r], u[r], h[r], q + QR * r, m + M * r); });
    if (dh_out.base != nullptr) {  // (alike for every thread)
      if (FULL && post) row_sum(reinterpret_cast<float(&)[M * R]>(m));
      each([&](int r, uint32_t i) { end(i, x[r], h[r], m + M * r, inverse1[r]); });
    }
    if constexpr (VEC) rows.done(R);
  };
  // One row at a time, whose last sums are taken with the next row's first ones: as many waits a
  // row as with two at a time, in fewer registers.
  const auto in_turn = [&] {
    Eight x, h;  // of the row before, until its dh
    float m[2] = {}, inverse1 = 1.0f;
    const bool late = post && dh_out.base != nullptr;
    for (uint32_t i = own.first; ; i += own.step) {
      const bool more = i < rows.rows, before = i != own.first;
      if (!more && !(late && before)) break;
      Eight nx, u, nh;
      float q[LAYER ? 8 : 4] = {};
      if (more) {
        if constexpr (VEC) rows.arrive();
        nx = rows.read(kInR, i, 1);
        u = rows.read(kInDy, i, 0);
        nh = rows.read(kInH, i, 2 + has_ds);
        if (layer || post_layer) {
          float mean[2] = {sum8(nx), sum8(nh)};
          row_sum(mean);
          center(nx, nh, mean);
        }
        products(nx, u, nh, q);
      }
#pragma unroll
      for (int k = 0; k < M; ++k) q[Q + k] = m[k];
      row_sum(q);
      if (late && before) end(i - own.step, x, h, q + Q, inverse1);
      if (!more) break;
      x = nx;
      h = nh;
      inverse1 = through(i, 0, x, u, h, q, m);
      if (!late && dh_out.base != nullptr) end(i, x, h, m, inverse1);
      if constexpr (VEC) rows.done();
    }
  };
  // With h, whose sums fill the registers, rows go in turn (8192 x 2048 45 us, one by one 47; 32768 x
  // 2048 137 and 148); where they are not asked for ahead, one by one, as their loads are what
  // counts (1003 x 775 15, in turn 20, two at a time 18).  Else two at a time (8192 x 2048 without
  // a norm after the block 28 us, one by one 41; 4096 x 8192, where a barrier is a cluster's, 125
  // and 177).
  if constexpr (FULL && VEC && SHARE == kBlock) {
    in_turn();
  } else {
    uint32_t i = own.first;
    if constexpr (!FULL || SHARE == kCluster)
      for (; i + own.step < rows.rows; i += 2 * own.step) make(std::integral_constant<int, 2>(), i);
    for (; i < rows.rows; i += own.step) make(std::integral_constant<int, 1>(), i);
  }
  const auto put = [&](int q, const Eight& x) {
    if ((a.wanted >> q & 1) == 0) return;
    float* to = a.sums + (static_cast<int64_t>(q) * a.blocks + own.first) * a.width;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      split(x.p[k], lo, hi);
      if (at.in(2 * k)) to[at.of(2 * k)] = lo;
      if (at.in(2 * k + 1)) to[at.of(2 * k + 1)] = hi;
    }
  };
  put(kDw, dw);
  if constexpr (LAYER) put(kDb, db);
  if constexpr (FULL) {
    const Eight g = at.load_vector(a.gate, 1.0f, wvec) * a.alpha;
    put(kDw1, ah * g);
    Eight dg = ah * w1.get();
    if constexpr (LAYER) {
      put(kDb1, aa * g);
      dg = fma8(aa, at.load_vector(a.b1, 0.0f, wvec), dg);
    }
    put(kDgate, dg * a.alpha);
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

// The blocks' sums in their order: 32 columns a block, 32 runs of blocks, which are added
// up in their order too.
constexpr int kRuns = 32;
__global__ void __launch_bounds__(32 * kRuns) block_norm_join_kernel(const __grid_constant__ NormJoinArgs a) {
  __shared__ float part[kRuns][33];
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
    for (int k = r; k < a.blocks; k += kRuns) sum += __ldcg(p + k * a.width);
  }
  part[r][c] = sum;
  __syncthreads();
  if (r != 0 || j >= a.width) return;
#pragma unroll
  for (int k = 1; k < kRuns; ++k) sum += part[k][c];
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

// Blocks (clusters) of the backward pass: 2 rows each at least (1, 2, 4, 8: 1003 x 775 15.7, 15.8,
// 21.4, 33 us; 2000 x 256 13.2, 7.7, 7.2, 7.5), and as many as are there at one time (512
// threads an SM).
int64_t backward_blocks(int64_t rows, int64_t width) {
  const RowShape r = row_shape(width);
  const int64_t n = (rows + 1) / 2;
  const int64_t most = kSms / r.cluster * (kMostThreads / r.threads);
  return n < most ? n : most;
}

uint32_t bytes_of(int64_t pitch) { return static_cast<uint32_t>(2 * pitch); }

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
  a.in[kInH] = L.h;
  a.s_out = L.s_out;
  a.y = L.y;
  a.dr = L.dr;
  a.dh = L.dh;
  a.pitch[kInGate] = bytes_of(s.ldg);
  a.pitch[kInH] = bytes_of(s.ldh);
  a.pitch_s = bytes_of(s.lds);
  a.pitch_y = bytes_of(s.ldy);
  a.pitch_dr = bytes_of(s.lddr);
  a.pitch_dh = bytes_of(s.lddh);
  a.pitch_dg = bytes_of(s.lddg);
  a.wvec = 1;
  for (const uint16_t* p : {a.w1, a.b1, a.w, a.b, a.gate})
    if (!aligned(p, 16)) a.wvec = 0;
  return a;
}

// Bytes of the ring, for each thread 16 of each input.
constexpr int kMostRing = kBackwardStages * kInputs * kMostThreads * 16;
static_assert(kMostRing + 8192 <= kSmem, "the ring and the parts of the sums");
int ring_bytes(const NormArgs& a, int threads, int stages) { return stages * a.inputs * threads * 16; }

// (Biases are LAYER's.)
bool has_layer(const NormArgs& a) { return a.kind == ZERO_NORM_LAYER || a.post == ZERO_NORM_LAYER; }

// Whether rows of every matrix lie on 16-byte boundaries; and how many inputs there are.
struct Rows16 {
  int64_t rows;
  bool all = true;
  void operator()(const void* p, uint32_t pitch) {
    if (p != nullptr && (!aligned(p, 16) || (rows > 1 && pitch % 16 != 0))) all = false;
  }
  explicit Rows16(NormArgs* a) : rows(a->rows) {
    for (int q = 0; q < kInputs; ++q) {
      (*this)(a->in[q], a->pitch[q]);
      if (a->in[q] != nullptr) ++a->inputs;
    }
  }
};

// A kernel with a ring of `smem` bytes.
template <typename Kernel>
cudaError_t launch_ring(Kernel kernel, int64_t blocks, int threads, int smem, int cluster, const NormArgs& a,
                        Chain* chain) {
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), kMostRing);
    if (e != cudaSuccess) return e;
  }
  return chain->launch(kernel, dim3(static_cast<unsigned>(blocks * cluster)), threads, smem, cluster, a);
}

template <bool FULL, bool LAYER>
cudaError_t launch_backward(const NormArgs& a, bool vec, Chain* chain) {
  const RowShape r = row_shape(a.width);
  const auto kernel = vec ? (r.cluster == 1 ? block_norm_backward_kernel<true, kBlock, FULL, LAYER>
                                            : block_norm_backward_kernel<true, kCluster, FULL, LAYER>)
                          : (r.cluster == 1 ? block_norm_backward_kernel<false, kBlock, FULL, LAYER>
                                            : block_norm_backward_kernel<false, kCluster, FULL, LAYER>);
  return launch_ring(kernel, a.blocks, r.threads, vec ? ring_bytes(a, r.threads, kBackwardStages) : 0, r.cluster, a, chain);
}

template <bool LAYER>
cudaError_t launch_forward(const NormArgs& a, bool vec, Chain* chain) {
  const RowShape r = row_shape(a.width);
  const int smem = vec ? ring_bytes(a, r.threads, kForwardStages) : 0;
  int64_t each = 1024 / r.threads;  // blocks an SM
  if (each > 24) each = 24;
  if (each > kSmem / (smem + 2560)) each = kSmem / (smem + 2560);
  const int64_t most = each * kSms / r.cluster;
  const auto kernel = vec ? (r.cluster == 1 ? block_norm_forward_kernel<true, kBlock, LAYER>
                                            : block_norm_forward_kernel<true, kCluster, LAYER>)
                          : (r.cluster == 1 ? block_norm_forward_kernel<false, kBlock, LAYER>
                                            : block_norm_forward_kernel<false, kCluster, LAYER>);
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
  a.pitch[kInR] = bytes_of(L.s.ldr);
  Rows16 vec(&a);
  vec(a.s_out, a.pitch_s);
  vec(a.y, a.pitch_y);
  Chain chain{L.stream};
  return has_layer(a) ? launch_forward<true>(a, vec.all, &chain) : launch_forward<false>(a, vec.all, &chain);
}

cudaError_t launch_block_norm_backward(const BlockNormLaunch& L) {
  (void)cudaGetLastError();
  NormArgs a = args_of(L);
  const bool one = L.s.ldg == 0;
  a.in[kInR] = L.sum;
  a.pitch[kInR] = bytes_of(L.s.lds);
  a.in[kInDy] = L.dy;
  a.pitch[kInDy] = bytes_of(L.s.lddy);
  a.in[kInDs] = L.ds;
  a.pitch[kInDs] = bytes_of(L.s.ldds);
  const bool full = L.h != nullptr && (a.post != ZERO_NORM_NONE || L.gate != nullptr);
  if (!full) a.in[kInH] = a.in[kInGate] = nullptr;  // (their values are not needed)
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
    vec(a.dr, a.pitch_dr);
    vec(a.dh, a.pitch_dh);
    vec(a.dgate_rows, a.pitch_dg);
    a.sums = static_cast<float*>(L.workspace);
    a.blocks = static_cast<int32_t>(backward_blocks(a.rows, a.width));
    const bool layer = has_layer(a);
    e = full ? (layer ? launch_backward<true, true>(a, vec.all, &chain)
                     : launch_backward<true, false>(a, vec.all, &chain))
             : (layer ? launch_backward<false, true>(a, vec.all, &chain)
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
  return chain.launch(block_norm_join_kernel, dim3(static_cast<unsigned>((a.width + 31) / 32), kinds),
                      32 * kRuns, 0, 1, j);
}

}  // namespace zeroadam
