// linear.cu -- a unit's linear maps, forward and backward, on sm_103a.
//
// The three products of a linear map are one, D[i,j] = sum over k of A(i,k)
// B(j,k), and differ in which way their operands lie in memory:
//   y  = x W^T     i: rows, j: out, k: in     A, B along k
//   dx = dz W      i: rows, j: in,  k: out    A along k, B along j
//   dw = dz^T x    i: out,  j: in,  k: rows   A along i, B along j
// The tensor cores take either way (K-major, MN-major) from tiles that TMA
// brings into shared memory, so no operand is transposed in memory.
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "linear_epilogue.cuh"
#include "linear_plan.hpp"
#include "train_ops.cuh"
#include "umma.cuh"

namespace zeroadam {
namespace {

// Status word of the products' bounded waits (read and cleared by
// zero_device_status): nonzero once a wait has given up.
__device__ int g_linear_status;
__device__ int g_linear_status_taken;

__global__ void take_linear_status_kernel() {
  g_linear_status_taken = atomicExch(&g_linear_status, 0);
}

struct ProductArgs {
  CUtensorMap a, b;
  CUtensorMap out, pre;  // D and pre, where e.vec
  CUtensorMap parts;     // [tail tile * splits + part][rows of a tile][bn], fp32
  Epilogue e;
  int64_t rows, cols;
  int32_t tiles_m, tiles_n, bn, a_rows;
  int32_t whole;         // tiles done in one piece
  int32_t splits;        // parts of the reduction of each tile after those
  int32_t steps;         // stages of the whole reduction
  int32_t withhold;      // test hook: no loads are issued, so every wait runs out
  int32_t late;          // its inputs were there before its predecessor began
  int32_t early_units;   // units that the predecessor leaves idle in its last round,
  int32_t early_tiles;   // and tiles they do meanwhile
};

struct Tile {
  int64_t row, col;  // of the tile's first element
  int first, last;   // stages
  int part;          // place in the parts, or -1: the whole reduction
};

// Item t of the work: the tiles in columns of up to 8 tiles of rows, so that the
// tiles in flight at one time share their operands in L2; after the first
// `whole` of them each tile is `splits` items, one for each part of the
// reduction, so that the last round of tiles keeps every SM busy.
__device__ __forceinline__ void part_of(const ProductArgs& a, int t, Tile& r) {
  r.part = -1;
  r.first = 0;
  r.last = a.steps;
  if (t >= a.whole && a.splits > 1) {
    r.part = t - a.whole;
    const int part = r.part % a.splits;
    r.first = static_cast<int>(static_cast<int64_t>(a.steps) * part / a.splits);
    r.last = static_cast<int>(static_cast<int64_t>(a.steps) * (part + 1) / a.splits);
  }
}
template <int BM>
__device__ __forceinline__ Tile tile_of(const ProductArgs& a, int t) {
  constexpr int kGroup = 8;
  Tile r;
  part_of(a, t, r);
  if (t >= a.whole) t = a.whole + (t - a.whole) / a.splits;
  const int group = t / (kGroup * a.tiles_n);
  const int m0 = group * kGroup;
  const int height = a.tiles_m - m0 < kGroup ? a.tiles_m - m0 : kGroup;
  const int in = t - group * kGroup * a.tiles_n;
  r.row = static_cast<int64_t>(m0 + in % height) * BM;
  r.col = static_cast<int64_t>(in / height) * a.bn;
  return r;
}

// Which epilogue a product has, settled when the kernel is compiled.
enum Kind {
  kForward,   // bias, pre, activation, residual; bf16
  kGradient,  // times an activation's slope, or added to what is there; bf16
  kFloat,     // fp32, alone or added to what is there
};

// A warp's 32 x 32 part of D from shared memory, where row r's 16-byte piece q
// (columns 4q to 4q+3) lies at piece q ^ (r & 7): bank conflicts neither where a
// lane writes its row nor where 4 or 8 lanes read one.
__device__ __forceinline__ int staged(int r, int q) { return r * 32 + ((q ^ (r & 7)) * 4); }

// Any layout, and the edges: a lane takes one column, 8 rows at a time so that
// their loads are under way together; whole eights have code of their own, without
// a predicate a row (fp32 dw of 8192 x 2047, 4096 rows: 150 us, else 173).
template <Kind KIND>
__device__ __noinline__ void epilogue_scalar(const Epilogue& e, const float* mine, int64_t row0,
                                             int64_t col0, int64_t rows, int64_t cols, int lane) {
  const int64_t j = col0 + lane;
  if (j >= cols) return;
  const int n = rows - row0 < 32 ? static_cast<int>(rows - row0) : 32;
  const bool accumulate = e.accumulate != 0;
  const int act = KIND == kForward ? e.act : e.slope_act;
  const int64_t ldo = e.ldo, ldp = e.ldp;
  const uint16_t* from = nullptr;
  int64_t from_pitch = 0;
  float bias = 0.0f;
  if constexpr (KIND == kForward) {
    from = e.residual;
    from_pitch = e.ldr;
    if (e.bias != nullptr) bias = bf16_at(e.bias + j);
  } else if constexpr (KIND == kGradient) {
    from = accumulate ? static_cast<const uint16_t*>(e.out) : e.slope_of;
    from_pitch = accumulate ? ldo : e.lds;
  }
  if (from != nullptr) from += row0 * from_pitch + j;
  float* out32 = static_cast<float*>(e.out) + row0 * ldo + j;
  uint16_t* out16 = static_cast<uint16_t*>(e.out) + row0 * ldo + j;
  uint16_t* pre = KIND == kForward && e.pre != nullptr ? e.pre + row0 * ldp + j : nullptr;
  const auto rows8 = [&](int r, auto all) {  // all: the 8 rows are there
    const auto each = [&](auto* p, int64_t pitch, auto f) {
#pragma unroll
      for (int k = 0; k < 8; ++k, p += pitch)
        if (all.value || r + k < n) f(k, p);
    };
    float x[8], y[8] = {};
    if (KIND == kFloat && accumulate) each(out32, ldo, [&](int k, float* p) { y[k] = *p; });
    if (KIND != kFloat && from != nullptr)
      each(from, from_pitch, [&](int k, const uint16_t* p) { y[k] = bf16_at(p); });
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = mine[32 * r + staged(k, lane / 4) + lane % 4] + bias;
    if (KIND == kForward) {
      if (pre != nullptr) each(pre, ldp, [&](int k, uint16_t* p) { *p = to_bf16(x[k]); });
      act_value8(x, act);
    }
    if (KIND == kGradient && !accumulate && from != nullptr) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        if (act == ZERO_ACT_GELU) times_slope2<ZERO_ACT_GELU>(x[k], x[k + 1], y[k], y[k + 1]);
        else if (act == ZERO_ACT_SILU) times_slope2<ZERO_ACT_SILU>(x[k], x[k + 1], y[k], y[k + 1]);
        else if (act == ZERO_ACT_RELU) times_slope2<ZERO_ACT_RELU>(x[k], x[k + 1], y[k], y[k + 1]);
      }
    } else if (KIND == kFloat ? accumulate : from != nullptr) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] += y[k];
    }
    if (KIND == kFloat) each(out32, ldo, [&](int k, float* p) { *p = x[k]; });
    else each(out16, ldo, [&](int k, uint16_t* p) { *p = to_bf16(x[k]); });
    out32 += 8 * ldo;
    out16 += 8 * ldo;
    if (pre != nullptr) pre += 8 * ldp;
    if (from != nullptr) from += 8 * from_pitch;
  };
#pragma unroll 1
  for (int r = 0; r < n; r += 8) {
    if (r + 8 <= n) rows8(r, std::true_type{});
    else rows8(r, std::false_type{});
  }
}

// 32 columns of fp32 as they are, in the room of both slots: no send() may
// follow (fp32 outputs have none, and split tiles are a unit's last).
__device__ __forceinline__ void send_sums(const CUtensorMap* map, uint8_t* staging,
                                          const float v[32], int x, int y, int z, bool sum,
                                          int lane) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<float4*>(staging + 4 * staged(lane, q)) =
        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  fence_async_shared();
  __syncwarp();
  if (lane == 0) {
    tile_store(map, staging, x, y, z, sum);
    bulk_commit();
  }
}

// A 32 x 32 part, a row a lane, through shared memory and out by TMA, which takes
// the addresses and the edges off the lanes and adds fp32 gradients to what is
// there itself, in L2 (128 x 8192 x 8192 fp32: 64 us with stores by the lanes, 56
// so; accumulating 138 and 115; what both come to below 2^-126 is 0 there).  A
// warp has 4 KB: two slots of bf16, or one of fp32, in TMA's swizzle, which keeps
// the lanes' 16-byte writes off each other's banks.
//
// The parameters are taken into registers once, and each step is one branch
// around its 32 columns: a warp runs a part alone, with nothing to hide a
// branch or a constant's load behind (a branch for each 8 columns, its pointer
// loaded anew, made a part 2,400 cycles).
template <Kind KIND>
struct EpiloguePart {
  const uint16_t *from, *bias_from;  // what it reads; NULL: nothing
  int64_t from_pitch;
  int32_t act;       // of the sum, or whose slope it is multiplied with
  bool pre, add;     // pre is written; what is read is added
  int slot = 0;
  uint4 in[4], bias[4];

  __device__ __forceinline__ explicit EpiloguePart(const Epilogue& e)
      : from(nullptr), bias_from(nullptr), from_pitch(0), act(ZERO_ACT_NONE), pre(false), add(true) {
    if constexpr (KIND == kForward) {
      from = e.residual;
      from_pitch = e.ldr;
      bias_from = e.bias;
      act = e.act;
      pre = e.pre != nullptr;
    } else if constexpr (KIND == kGradient) {
      add = e.accumulate != 0;
      from = add ? static_cast<const uint16_t*>(e.out) : e.slope_of;
      from_pitch = add ? e.ldo : e.lds;
      act = e.slope_act;
    } else {
      add = e.accumulate != 0;
    }
  }
  // Asks for what the part reads, before its sums are there.
  __device__ __forceinline__ void ask(int64_t row, int64_t col, bool mine) {
    if constexpr (KIND != kFloat) {
      if (from != nullptr && mine) {
        const uint4* p = reinterpret_cast<const uint4*>(from + row * from_pitch + col);
#pragma unroll
        for (int q = 0; q < 4; ++q) in[q] = p[q];
      }
      if (KIND == kForward && bias_from != nullptr) {
        const uint4* p = reinterpret_cast<const uint4*>(bias_from + col);
#pragma unroll
        for (int q = 0; q < 4; ++q) bias[q] = __ldg(p + q);
      }
    }
  }
  // 32 columns of bf16 into a slot and off.
  __device__ __forceinline__ void send(const CUtensorMap* map, uint8_t* staging, const float v[32],
                                       int x, int y, int lane) {
    if (lane == 0) bulk_wait_read<1>();  // the copy before the last has left this slot
    __syncwarp();
    uint8_t* to = staging + 2048 * slot;
    slot ^= 1;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(to + lane * 64 + ((q ^ ((lane >> 1) & 3)) * 16)) = to_bf16x8(v + 8 * q);
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      tile_store(map, to, x, y, 0, false);
      bulk_commit();
    }
  }
  __device__ __forceinline__ static void plus(float v[32], const uint4 w[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float y[8];
      bf16x8(w[q], y);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[8 * q + c] += y[c];
    }
  }
  template <int ACT>
  __device__ __forceinline__ void times_slope(float v[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float z[8];
      bf16x8(in[q], z);
#pragma unroll
      for (int c = 0; c < 8; c += 2)
        times_slope2<ACT>(v[8 * q + c], v[8 * q + c + 1], z[c], z[c + 1]);
    }
  }
  template <int ACT>
  __device__ __forceinline__ static void activate(float v[32]) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) act_value2<ACT>(v[c], v[c + 1]);
  }
  __device__ __forceinline__ void put(const ProductArgs& a, uint8_t* staging, float v[32], int row,
                                      int col, int lane) {
    if constexpr (KIND == kFloat) {
      send_sums(&a.out, staging, v, col, row, 0, add, lane);
    } else {
      if constexpr (KIND == kForward) {
        if (bias_from != nullptr) plus(v, bias);
        if (pre) send(&a.pre, staging, v, col, row, lane);
        if (act == ZERO_ACT_GELU) activate<ZERO_ACT_GELU>(v);
        else if (act == ZERO_ACT_SILU) activate<ZERO_ACT_SILU>(v);
        else if (act == ZERO_ACT_RELU) activate<ZERO_ACT_RELU>(v);
      }
      if (from != nullptr) {
        if (KIND == kForward || add) plus(v, in);
        else if (act == ZERO_ACT_GELU) times_slope<ZERO_ACT_GELU>(v);
        else if (act == ZERO_ACT_SILU) times_slope<ZERO_ACT_SILU>(v);
        else if (act == ZERO_ACT_RELU) times_slope<ZERO_ACT_RELU>(v);
      }
      send(&a.out, staging, v, col, row, lane);
    }
  }
};

// The same for bf16 matrices that TMA cannot write: rows begin anywhere (odd
// pitches, offsets).  A lane's row begins s elements (0 to 7) past a 16-byte
// boundary in every part of a tile, as parts are 32 columns and a warp's lie side
// by side; so a part is moved up by s, behind the last s columns of the part to
// its left, and goes in aligned vectors, 4 lanes a row.  What is left at both ends
// of a warp's columns goes in pieces of 2, 4 and 8 bytes.  8192 x 768 -> 50257: 462
// us (50304 columns, by TMA: 376; a column a lane, 2 bytes at a time: 909); with
// bias and residual 895 (2,562 so); what bounds it is the warps' instructions, some
// 250 a part.
template <Kind KIND>
struct RowsPart {
  const uint16_t *from, *bias;
  uint16_t *out, *pre;
  int64_t from_pitch, out_pitch, pre_pitch;
  int32_t act;
  bool add;
  uint32_t in[20];  // what the part reads, from the vector on that its first column is in
  float b;          // the lane's column's bias
  uint4 before_out, before_pre;  // the part to the left: its last 8 columns

  __device__ __forceinline__ explicit RowsPart(const Epilogue& e)
      : from(nullptr), bias(nullptr), out(static_cast<uint16_t*>(e.out)), pre(nullptr),
        from_pitch(0), out_pitch(e.ldo), pre_pitch(0), act(ZERO_ACT_NONE), add(true), b(0.0f) {
    if constexpr (KIND == kForward) {
      from = e.residual;
      from_pitch = e.ldr;
      bias = e.bias;
      act = e.act;
      pre = e.pre;
      pre_pitch = e.ldp;
    } else {
      add = e.accumulate != 0;
      from = add ? out : e.slope_of;
      from_pitch = add ? out_pitch : e.lds;
      act = e.slope_act;
    }
  }
  // Elements from the 16-byte boundary before p to it.
  __device__ __forceinline__ static int past(const uint16_t* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) / 2 % 8);
  }
  // o: elements `first` (0 to 8) on of v.
  template <int N, int M>
  __device__ __forceinline__ static void moved(uint32_t (&v)[N], int first, uint32_t (&o)[M]) {
#pragma unroll
    for (int k = 4; k >= 1; k /= 2)
#pragma unroll
      for (int i = 0; i < M + k && i + k < N; ++i) v[i] = (first / 2) & k ? v[i + k] : v[i];
#pragma unroll
    for (int i = 0; i < M; ++i)
      o[i] = __funnelshift_r(v[i], i + 1 < N ? v[i + 1] : 0u, 16 * (first & 1));
  }
  // Asks for what the part at `col` reads; the warp's columns are [first, end).
  __device__ __forceinline__ void ask(int64_t row, int64_t col, bool mine, int64_t first,
                                      int64_t end, int lane) {
    if (KIND == kForward && bias != nullptr)
      b = col + lane < end ? bf16_at(bias + col + lane) : 0.0f;
    if (from == nullptr || !mine) return;
    const uint16_t* at = from + row * from_pitch + col;
    const int s = past(at);
    at -= s;
    const int low = static_cast<int>(first - col) + s, high = static_cast<int>(end - col) + s;
    const int stop = high < 32 + s ? high : 32 + s;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (8 * k >= low && 8 * k + 8 <= high) {
        x = *reinterpret_cast<const uint4*>(at + 8 * k);
      } else if (8 * k < stop) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (8 * k + q >= low && 8 * k + q < stop)
            w[q / 2] |= static_cast<uint32_t>(at[8 * k + q]) << (16 * (q % 2));
        x = make_uint4(w[0], w[1], w[2], w[3]);
      }
      in[4 * k] = x.x; in[4 * k + 1] = x.y; in[4 * k + 2] = x.z; in[4 * k + 3] = x.w;
    }
  }
  // 32 columns into rows of p, from `col` on.
  __device__ __forceinline__ void send(uint16_t* p, int64_t pitch, uint4& before, uint4* staging,
                                       const float x[32], int64_t row0, int64_t rows, int64_t col,
                                       int64_t first, int64_t end, int lane) {
    uint16_t* at = p + (row0 + lane) * pitch + col;
    const int s = past(at);
    uint32_t v[25], o[20];
    v[0] = before.x; v[1] = before.y; v[2] = before.z; v[3] = before.w;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[4 + i] = bf16x2_bits(x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 20; i < 25; ++i) v[i] = 0;
    before = make_uint4(v[16], v[17], v[18], v[19]);
    moved(v, 8 - s, o);
    __syncwarp();  // the part before has been read
#pragma unroll
    for (int q = 0; q < 4; ++q)
      staging[lane * 4 + (q ^ (lane / 2 % 4))] =
          make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    __syncwarp();
    const int low = static_cast<int>(first - col), high = static_cast<int>(end - col);
    const int i0 = lane / 4, q = lane % 4, n = rows - row0 < 32 ? static_cast<int>(rows - row0) : 32;
    uint16_t* to = p + (row0 + i0) * pitch + col + 8 * q;
#pragma unroll
    for (int k = 0; k < 4; ++k, to += 8 * pitch) {
      const int c = 8 * q - past(to);
      if (8 * k + i0 < n && c >= low && c + 8 <= high)
        *reinterpret_cast<uint4*>(to - past(to)) = staging[(8 * k + i0) * 4 + (q ^ (i0 / 2 % 4))];
    }
    if (lane >= n) return;
    at -= s;
    if (low == 0 && s > 0) {
      int j = s;
      if (j & 1) {
        const uint32_t w = j == 1 ? o[0] : j == 3 ? o[1] : j == 5 ? o[2] : o[3];
        at[j++] = static_cast<uint16_t>(w >> 16);
      }
      if (j & 2) {
        *reinterpret_cast<uint32_t*>(at + j) = j == 2 ? o[1] : o[3];
        j += 2;
      }
      if (j & 4) *reinterpret_cast<uint2*>(at + 4) = make_uint2(o[2], o[3]);
    }
    const int left = (s + high) % 8;
    if (high <= 32 && left > 0) {
      const int k = (s + high) / 8;
      const uint4 w = k < 4 ? staging[lane * 4 + (k ^ (lane / 2 % 4))]
                            : make_uint4(o[16], o[17], o[18], o[19]);
      at += 8 * k;
      if (left & 4) *reinterpret_cast<uint2*>(at) = make_uint2(w.x, w.y);
      if (left & 2) *reinterpret_cast<uint32_t*>(at + (left & 4)) = left & 4 ? w.z : w.x;
      if (left & 1)
        at[left - 1] = static_cast<uint16_t>(left == 1 ? w.x : left == 3 ? w.y : left == 5 ? w.z : w.w);
    }
  }
  template <typename F>
  __device__ __forceinline__ static void pairs(float x[32], const uint32_t w[16], F f) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      f(x[2 * i], x[2 * i + 1], __uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  // At least 8 columns are the warp's.
  __device__ __forceinline__ void put(float* mine, float x[32], int64_t row0, int64_t rows,
                                      int64_t col, int64_t first, int64_t end, int lane) {
    uint4* staging = reinterpret_cast<uint4*>(mine);
    if constexpr (KIND == kForward) {
      if (bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] += __shfl_sync(0xffffffffu, b, i);
      }
      if (pre != nullptr)
        send(pre, pre_pitch, before_pre, staging, x, row0, rows, col, first, end, lane);
      if (act == ZERO_ACT_GELU) EpiloguePart<KIND>::template activate<ZERO_ACT_GELU>(x);
      else if (act == ZERO_ACT_SILU) EpiloguePart<KIND>::template activate<ZERO_ACT_SILU>(x);
      else if (act == ZERO_ACT_RELU) EpiloguePart<KIND>::template activate<ZERO_ACT_RELU>(x);
    }
    if (from != nullptr) {
      uint32_t w[16];
      moved(in, past(from + (row0 + lane) * from_pitch + col), w);
      if (add)
        pairs(x, w, [](float& a, float& b, float c, float d) { a += c; b += d; });
      else if (act == ZERO_ACT_GELU)
        pairs(x, w, [](float& a, float& b, float c, float d) {
          times_slope2<ZERO_ACT_GELU>(a, b, c, d);
        });
      else if (act == ZERO_ACT_SILU)
        pairs(x, w, [](float& a, float& b, float c, float d) {
          times_slope2<ZERO_ACT_SILU>(a, b, c, d);
        });
      else if (act == ZERO_ACT_RELU)
        pairs(x, w, [](float& a, float& b, float c, float d) {
          times_slope2<ZERO_ACT_RELU>(a, b, c, d);
        });
    }
    send(out, out_pitch, before_out, staging, x, row0, rows, col, first, end, lane);
  }
};

// Place in the ring of stages: the stage, and the parity of its barriers' phase.
struct Place {
  int stages;
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Place(int n) : stages(n) {}
  __device__ __forceinline__ void next() {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// Stages that are summed in tensor memory before the sum is taken over in fp32.
// The tensor cores cut off what does not fit a sum's 24 bits, so a chain of
// additions comes out too small by 1e-9 of itself for each step of the reduction
// (1e-6 over 1,024 steps, 4e-6 over 4,096).  fp32 gradients are worth more than
// that: their chains end after 768 steps, and the epilogue's warps add them up in
// registers, rounding to nearest.  Results in bf16 keep one chain: its loss is
// below a hundredth of their rounding up to 16,384 steps.
template <Kind KIND>
constexpr int kChain = KIND == kFloat ? 768 / kStep : INT32_MAX;

// A wait for a chain, which may take `stages` stages: 1 s, and 10 us for each.
__device__ __forceinline__ bool wait_for_chain(uint64_t* bar, uint32_t parity, int stages) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t limit = kWaitLimitNs + static_cast<uint64_t>(stages) * 10000u, t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > limit) return false;
  return true;
}

// Persistent and specialised by warp.  Warp 0 brings the operands' tiles into a
// ring of stages; warp 1 of the tile's first CTA issues the matrix
// instructions, accumulating in one half of tensor memory while the other
// warps take the tile before it out of the other half, through the epilogue.
// Barriers: full[s] (in the first CTA) counts the bytes of both CTAs' loads of
// stage s; empty[s] (in both) is arrived on when the products that read it are
// done; done[b] (in both) when half b holds a finished tile; free_[b] (in the
// first CTA) when every epilogue warp has read it.
// Every wait is bounded; one that gives up sets g_linear_status and ends its
// warp's loop, and the others' waits then run out too.
// What bounds it is the tensor cores: at 8192^3 a stage takes 1,039 cycles where
// its matrix instructions alone are 1,024 (1,922 TFLOP/s, 572 us); at 8192 x 2048
// x 8192, 154 us, 14 rounds of tiles where 13.47 are needed, and 8 us of beginning
// and end.
// ROWS: D, pre or what is read with them lies where TMA cannot take it.
//
// GATHER: a cluster's CTAs have a part of one tile's reduction each, and no other
// item.  They leave their sums in the ring, which nothing is loaded into any more,
// and each adds up every splits-th 32 columns of all, in the parts' order.  For few
// tiles: an SM takes in some 60 bytes a cycle whatever the tile, so more SMs with
// less of the reduction each are faster, by more than the exchange costs (256 x 4096
// -> 4096 17.4 -> 14.8 us, 300 x 4096 -> 1024 12.6 -> 11.1, 64 x 11008 -> 4096 23.5 ->
// 21.6; 128 x 4096 -> 4096 with the parts through global memory and joined by a
// launch 14.7, 13.7 so).
template <int CG, bool A_MN, bool B_MN, Kind KIND, bool ROWS, bool GATHER>
__global__ void __launch_bounds__(kProductThreads, 1)
    linear_product_kernel(const __grid_constant__ ProductArgs a) {
  using Shape = ProductShape<CG>;
  constexpr int BM = CG * kBlockRows;
  const int b_rows = a.bn / CG, pair = pair_bytes(a.a_rows, b_rows), stage = kSub * pair;
  const int stages = ring_stages(a.a_rows, b_rows), a_bytes = a.a_rows * kDepth * 2;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  float* staging = reinterpret_cast<float*>(ring + stages * stage);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + stages * stage + kStaging);
  uint64_t* empty = full + kMaxStages;
  uint64_t* done = empty + kMaxStages;
  uint64_t* free_ = done + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(free_ + 2);
  uint32_t* failed = tmem_at + 1;  // GATHER: this CTA's sums are not there

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int unit = blockIdx.x / CG;
  const Turns turns{a.early_units, a.early_tiles, static_cast<int>(gridDim.x) / CG};
  const int tiles = a.whole + (a.tiles_m * a.tiles_n - a.whole) * a.splits;

  if (threadIdx.x == 0) {
    *failed = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&done[b], 1);
      mbar_init(&free_[b], kEpilogueWarps * CG);
    }
    mbar_init_fence();
  }
  if (threadIdx.x == 64) {
    prefetch_map(&a.a);
    prefetch_map(&a.b);
  }
  if (warp == 1) tmem_alloc<CG>(tmem_at, Shape::kColumns);
  if (!a.late) wait_for_predecessor();
  launch_dependents();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp == 0) {
    if (lane == 0) {
      Place at(stages);
      int issued = 0;  // stages, up to the ring's
      bool ok = true;
      Tile next = tile_of<BM>(a, turns.first(unit));
      for (int t = turns.first(unit); t < tiles && ok; t = turns.after(t)) {
        const Tile tile = next;
        const int ra = static_cast<int>(tile.row) + rank * kBlockRows;
        const int rb = static_cast<int>(tile.col) + rank * b_rows;
        for (int step = tile.first; step < tile.last; ++step, at.next()) {
          if (issued == stages) {
            if (!mbar_wait(&empty[at.s], at.phase ^ 1)) {
              ok = false;
              break;
            }
          } else {
            ++issued;
          }
          if (a.withhold) {
            if (step == tile.first && turns.after(t) < tiles) next = tile_of<BM>(a, turns.after(t));
            continue;
          }
          const uint32_t bar = CG == 2 ? peer_addr(&full[at.s], 0) : smem_addr(&full[at.s]);
          if (rank == 0) mbar_expect_tx(&full[at.s], CG * stage);
#pragma unroll
          for (int h = 0; h < kSub; ++h) {
            uint8_t* sa = ring + at.s * stage + h * pair;
            uint8_t* sb = sa + a_bytes;
            const int x = step * kStep + h * kDepth;
            if constexpr (A_MN) {
#pragma unroll
              for (int c = 0; c < kBlockRows / 64; ++c)
                tile_load<CG>(sa + c * 64 * kDepth * 2, &a.a, ra + 64 * c, x, bar);
            } else {
              tile_load<CG>(sa, &a.a, x, ra, bar);
            }
            if constexpr (B_MN) {
              for (int c = 0; c < b_rows / 64; ++c)
                tile_load<CG>(sb + c * 64 * kDepth * 2, &a.b, rb + 64 * c, x, bar);
            } else {
              tile_load<CG>(sb, &a.b, x, rb, bar);
            }
          }
          // (off the path from one tile's last loads to the next one's first)
          if (step == tile.first && turns.after(t) < tiles) next = tile_of<BM>(a, turns.after(t));
        }
      }
      if (!ok) atomicExch(&g_linear_status, 1);
      // No CTA ends while loads into it, or arrivals on its barriers, are under
      // way: the products that read the last stages are waited for.
      if (!a.withhold) {
        if (issued < stages) at = Place(stages);
        for (int j = 0; j < issued; ++j, at.next()) {
          // stage at.s was filled last in the phase before this place's, or, in a
          // ring not yet full, in its first
          const uint32_t phase = issued < stages ? at.phase : at.phase ^ 1;
          mbar_wait(&empty[at.s], phase);
          if (!ok && rank == 0) mbar_wait(&full[at.s], phase);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t desc = mma_desc(BM, a.bn, A_MN, B_MN);
      // bytes between two steps of 16 of the reduction, and the distances of
      // smem_desc, along each operand's rows
      constexpr uint32_t step_a = A_MN ? 16 * 128 : 32, step_b = B_MN ? 16 * 128 : 32;
      constexpr uint32_t lead = 64 * kDepth * 2, stride = 1024;
      Place at(stages);
      int used = 0;  // stages, up to the ring's
      int n = 0;     // chains begun
      bool ok = true;
      for (int t = turns.first(unit); t < tiles && ok; t = turns.after(t)) {
        Tile tile;
        part_of(a, t, tile);
        for (int step = tile.first; step < tile.last && ok; ++n) {
          const int first = step;
          const int last = tile.last - step > kChain<KIND> ? step + kChain<KIND> : tile.last;
          const int b = n & 1;
          if (n >= 2 && !mbar_wait(&free_[b], static_cast<uint32_t>((n / 2 - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (; step < last; ++step, at.next()) {
            if (!mbar_wait(&full[at.s], at.phase)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (used < stages) ++used;
#pragma unroll
            for (int h = 0; h < kSub; ++h) {
              const uint32_t sa = smem_addr(ring) + at.s * stage + h * pair;
              const uint64_t da = smem_desc(sa, lead, stride);
              const uint64_t db = smem_desc(sa + a_bytes, lead, stride);
#pragma unroll
              for (int q = 0; q < kDepth / 16; ++q)
                mma_bf16<CG>(tmem + b * Shape::kMaxCols, da + q * (step_a >> 4),
                             db + q * (step_b >> 4), desc, step > first || q > 0 || h > 0);
            }
            mma_commit<CG>(&empty[at.s]);
          }
          if (ok) mma_commit<CG>(&done[b]);
        }
      }
      if (!ok) {
        // products already issued end before tensor memory is freed
        atomicExch(&g_linear_status, 2);
        if (used < stages) at = Place(stages);
        for (int j = 0; j < used; ++j, at.next())
          mbar_wait(&empty[at.s], used < stages ? at.phase : at.phase ^ 1);
      }
    }
  } else {
    const int quarter = warp % 4, half = (warp - 2) / 4;
    float* mine = staging + (warp - 2) * 32 * 32;
    std::conditional_t<ROWS, RowsPart<KIND>, EpiloguePart<KIND>> part(a.e);
    const bool vec = a.e.vec != 0;
    const int bn = a.bn;
    // The columns of a tile that are this warp's, 32 at a time: every other 32, or half
    // of all.  Halves are what RowsPart needs; with them the gradient's reads of what
    // is there are faster (8192 x 8192 x 128 times a slope: 99 us, else 121), the
    // forward's writes slower (8192 x 128 x 8192: 58, else 52; plus a residual 105, 93).
    constexpr bool kBeside = ROWS || KIND == kGradient;
    const int c_first = 32 * half * (kBeside ? (bn / 32 + 1) / 2 : 1);
    const int c_end = kBeside && half == 0 ? (bn / 32 + 1) / 2 * 32 : bn;
    constexpr int c_step = kBeside ? 32 : 64;
    const int64_t rows = a.rows, cols = a.cols;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // This half of tensor memory has been read by the warp and may be written again.
    const auto release = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_peer(peer_addr(&free_[b], 0));
        else mbar_arrive(&free_[b]);
      }
    };
    int n = 0;
    bool ok = true;
    for (int t = turns.first(unit); t < tiles && ok; t = turns.after(t)) {
      const Tile tile = tile_of<BM>(a, t);
      const int64_t row0 = tile.row + rank * kBlockRows + quarter * 32;
      // (rows past the end are left out by the copy)
      const bool any = row0 < rows;
      const int64_t first = tile.col + c_first, end = tile.col + c_end < cols ? tile.col + c_end : cols;
      const bool fast = any && tile.part < 0 &&
                        (ROWS ? end - first >= 8 : vec && tile.col + bn <= cols);
      const bool mine_in = row0 + lane < rows;
      const auto ask = [&](int c) {
        if constexpr (ROWS) {
          if (tile.col + c < end) part.ask(row0 + lane, tile.col + c, mine_in, first, end, lane);
        } else {
          part.ask(row0 + lane, tile.col + c, mine_in);
        }
      };
      // 32 columns from c on are summed up: on their way.
      const auto finish = [&](float x[32], int c) {
        const int64_t col0 = tile.col + c;
        if constexpr (GATHER) {
          float* to = reinterpret_cast<float*>(ring) + (c / 32 * 4 + quarter) * 32 * 32;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(to + staged(lane, q)) =
                make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          return;
        }
        if constexpr (ROWS) {
          if (fast) {
            if (col0 < end) part.put(mine, x, row0, rows, col0, first, end, lane);
            return;
          }
        } else if (fast) {
          part.put(a, reinterpret_cast<uint8_t*>(mine), x, static_cast<int>(row0),
                   static_cast<int>(col0), lane);
          return;
        }
        if (!any || col0 >= cols) return;
        if (tile.part >= 0) {
          send_sums(&a.parts, reinterpret_cast<uint8_t*>(mine), x, c,
                    static_cast<int>(row0 - tile.row), tile.part, false, lane);
          return;
        }
        if constexpr (!ROWS) {
          if (vec && col0 + 32 <= cols) {
            part.ask(row0 + lane, col0, mine_in);
            part.put(a, reinterpret_cast<uint8_t*>(mine), x, static_cast<int>(row0),
                     static_cast<int>(col0), lane);
            return;
          }
        }
        {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(mine + staged(lane, q)) =
                make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          __syncwarp();
          epilogue_scalar<KIND>(a.e, mine, row0, col0, rows, cols, lane);
          __syncwarp();
        }
      };
      if constexpr (KIND == kFloat) {
        constexpr int kParts = Shape::kMaxCols / 64;
        float sum[kParts][32];
        for (int step = tile.first; step < tile.last; step += kChain<KIND>, ++n) {
          const int b = n & 1;
          ok = wait_for_chain(&done[b], static_cast<uint32_t>((n / 2) & 1), kChain<KIND>);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            const int c = c_first + c_step * i;
            if (c >= c_end) break;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {  // 16 at a time: 128 registers hold the sums
              uint32_t bits[16];
              tmem_load16(lanes + b * Shape::kMaxCols + c + h, bits);
              tmem_load_wait();
              if (step == tile.first) {
#pragma unroll
                for (int q = 0; q < 16; ++q) sum[i][h + q] = __uint_as_float(bits[q]);
              } else {
#pragma unroll
                for (int q = 0; q < 16; ++q) sum[i][h + q] += __uint_as_float(bits[q]);
              }
            }
          }
          release(b);
        }
        if (ok) {
#pragma unroll
          for (int i = 0; i < kParts; ++i)
            if (c_first + c_step * i < c_end) finish(sum[i], c_first + c_step * i);
        }
      } else {
        const int b = n & 1;
        ok = wait_for_chain(&done[b], static_cast<uint32_t>((n / 2) & 1), tile.last - tile.first);
        ++n;
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = lanes + b * Shape::kMaxCols;
        uint32_t bits[32];
        if (c_first < c_end) {
          tmem_load32(from + c_first, bits);
          if (fast) ask(c_first);
        } else {
          release(b);  // nothing of a tile this narrow is this warp's
        }
#pragma unroll 1
        for (int c = c_first; c < c_end; c += c_step) {
          float x[32];
          tmem_load_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q) x[q] = __uint_as_float(bits[q]);
          // the next part's sums come while this one's are worked on
          if (c + c_step < c_end) tmem_load32(from + c + c_step, bits);
          else release(b);
          finish(x, c);
          if (fast && c + c_step < c_end) ask(c + c_step);
        }
      }
    }
    if (!ok && lane == 0) {
      atomicExch(&g_linear_status, 3);
      if (GATHER) *failed = 1;
    }
    if (!GATHER && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  if constexpr (GATHER) {
    cluster_sync_writes();
    if (warp >= 2) {
      const int quarter = warp % 4, half = (warp - 2) / 4, mine_of = static_cast<int>(cluster_rank());
      float* mine = staging + (warp - 2) * 32 * 32;
      bool ok = true;
      for (int s = 0; s < a.splits; ++s)
        ok = ok && peer_load_u32(peer_addr(failed, s)) == 0;
      const Tile tile = tile_of<BM>(a, unit);
      const int64_t row0 = tile.row + quarter * 32;
      std::conditional_t<ROWS, RowsPart<KIND>, EpiloguePart<KIND>> part(a.e);
      for (int c = 32 * (mine_of + a.splits * half); c < a.bn; c += 64 * a.splits) {
        const int64_t col0 = tile.col + c;
        if (!ok || row0 >= a.rows || col0 >= a.cols) break;
        const int64_t end = a.cols < col0 + 32 ? a.cols : col0 + 32;
        const bool whole = ROWS ? end - col0 >= 8 : a.e.vec && col0 + 32 <= a.cols;
        if (whole) {
          if constexpr (ROWS) part.ask(row0 + lane, col0, row0 + lane < a.rows, col0, end, lane);
          else part.ask(row0 + lane, col0, row0 + lane < a.rows);
        }
        const float* from = reinterpret_cast<const float*>(ring) + (c / 32 * 4 + quarter) * 32 * 32;
        // A load takes 4 whole rows, two parts at a time (16 bytes of 32 rows, a row a
        // lane, made the kernel 22 us instead of 16 at 128 x 4096 -> 4096).
        float4 sum[8] = {};
#pragma unroll 1
        for (int s = 0; s < a.splits; s += 2) {
          float4 y[16];
#pragma unroll
          for (int q = 0; q < 16; ++q)
            y[q] = peer_load(peer_addr(from, s + q / 8) + 4 * staged(4 * (q % 8) + lane / 8, lane % 8));
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            float4& t = sum[q % 8];
            t.x += y[q].x; t.y += y[q].y; t.z += y[q].z; t.w += y[q].w;
          }
        }
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(mine + staged(4 * q + lane / 8, lane % 8)) = sum[q];
        __syncwarp();
        if (whole) {
          float x[32];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 y = *reinterpret_cast<const float4*>(mine + staged(lane, q));
            x[4 * q] = y.x; x[4 * q + 1] = y.y; x[4 * q + 2] = y.z; x[4 * q + 3] = y.w;
          }
          __syncwarp();
          if constexpr (ROWS)
            part.put(mine, x, row0, a.rows, col0, col0, end, lane);
          else
            part.put(a, reinterpret_cast<uint8_t*>(mine), x, static_cast<int>(row0),
                     static_cast<int>(col0), lane);
        } else {
          epilogue_scalar<KIND>(a.e, mine, row0, col0, a.rows, a.cols, lane);
          __syncwarp();
        }
      }
      if (lane == 0) bulk_wait_all();
      __syncwarp();
    }
  }
  __syncthreads();
  if constexpr (CG == 2 || GATHER) cluster_sync();
  if (warp == 1) tmem_free<CG>(tmem, Shape::kColumns);
  // what follows this kernel follows its predecessor too
  if (a.late) wait_for_predecessor();
}

// The parts of the tiles whose reduction was split, added in their order, and the
// epilogue: 8 columns a thread.
template <int BM>
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ ProductArgs a,
                                                          const float* parts) {
  const int per_row = a.bn / 8;
  const int u = blockIdx.y;  // of the tiles split
  const Tile tile = tile_of<BM>(a, a.whole + u * a.splits);
  const int in = blockIdx.x * 256 + threadIdx.x;
  const int r = in / per_row, c = in % per_row * 8;
  const int64_t i = tile.row + r, j = tile.col + c;
  wait_for_predecessor();
  launch_dependents();
  if (r >= BM || i >= a.rows || j >= a.cols) return;
  const Epilogue& e = a.e;
  const bool vec = e.vec && j + 8 <= a.cols;
  float x[8] = {};
  const float* p = parts + (static_cast<int64_t>(u) * a.splits * BM + r) * a.bn + c;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s, p += BM * a.bn) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
    const float4 w = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w;
    x[4] += w.x; x[5] += w.y; x[6] += w.z; x[7] += w.w;
  }
  if (!vec || e.out_f32) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (j + k < a.cols) epilogue_element(e, i, j + k, x[k]);
    return;
  }
  float y[8];
  auto add = [&](const uint16_t* from) {
    bf16x8(*reinterpret_cast<const uint4*>(from), y);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] += y[k];
  };
  if (e.bias != nullptr) add(e.bias + j);
  if (e.pre != nullptr) *reinterpret_cast<uint4*>(e.pre + i * e.ldp + j) = to_bf16x8(x);
  act_value8(x, e.act);
  if (e.residual != nullptr) add(e.residual + i * e.ldr + j);
  if (e.slope_of != nullptr)
    times_slope8(x, *reinterpret_cast<const uint4*>(e.slope_of + i * e.lds + j), e.slope_act);
  uint16_t* o = static_cast<uint16_t*>(e.out) + i * e.ldo + j;
  if (e.accumulate) add(o);
  *reinterpret_cast<uint4*>(o) = to_bf16x8(x);
}

// ------------------------------------------------------------------ layouts

bool aligned(const void* p, uintptr_t k) { return (reinterpret_cast<uintptr_t>(p) & (k - 1)) == 0; }

// A bf16 matrix as it lies in memory.  A single row has no pitch.
struct Stored {
  const uint16_t* p;
  int64_t rows, cols, ld;
  Stored() = default;
  Stored(const uint16_t* p, int64_t rows, int64_t cols, int64_t ld)
      : p(p), rows(rows), cols(cols), ld(rows > 1 ? ld : round_up(cols, 8)) {}
};

// Whether TMA can read it in place.
bool tileable(const Stored& m) { return aligned(m.p, 16) && m.ld % 8 == 0; }
// Pitch and bytes of a copy: rows on 128-byte boundaries, one swizzled row of
// TMA's each (with rows on odd multiples of 16 bytes its loads take twice the
// time: 1003 x 776 x 2312 backward 21 to 26 us a product).
int64_t copy_pitch(int64_t cols) { return round_up(cols, 64); }
int64_t copy_bytes(const Stored& m) { return round_up(m.rows * copy_pitch(m.cols) * 2, 256); }

struct CopyArgs {
  const uint16_t* src;
  uint16_t* dst;
  int64_t rows, cols, lds, ldd;
};
// dbias from the column sums of `blocks` blocks of rows.
struct DbiasArgs {
  const float* sums;  // [blocks][cols rounded up to 4]
  int64_t cols;
  int32_t blocks;
  void* dbias;        // NULL: not wanted
  int32_t out_f32, accumulate;
};

struct PrepareArgs {
  CopyArgs copy[3];
  int32_t copies;
  DbiasArgs dbias;
};

// A matrix laid out anew with rows on 128-byte boundaries.  A lane writes 16
// bytes of a row; it reads the aligned 16 bytes in which they begin, takes those
// in which they end from its neighbour, and shifts.  Vectors that lie partly
// outside the matrix's memory are read element by element.
__device__ __forceinline__ uint4 aligned_load(const char* p, const char* begin, const char* end) {
  if (p >= begin && p + 16 <= end) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {};
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (p + 2 * c >= begin && p + 2 * c < end)
      w[c / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p + 2 * c)))
                  << (16 * (c & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void copy_rows(const CopyArgs& a) {
  const int64_t per = (a.cols + 255) / 256;  // warps a row
  const int lane = threadIdx.x % 32;
  const char* begin = reinterpret_cast<const char*>(a.src);
  const char* end = begin + 2 * ((a.rows - 1) * a.lds + a.cols);
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; q < a.rows * per;
       q += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t i = q / per, j0 = (q - i * per) * 256;
    const char* s = begin + 2 * (i * a.lds + j0);
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s)) & 15u;
    s += 16 * lane - static_cast<int>(off);
    const uint4 u = aligned_load(s, begin, end);
    uint32_t w[9] = {u.x, u.y, u.z, u.w, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) w[4 + k] = __shfl_down_sync(0xffffffffu, w[k], 1);
    if (lane == 31 && off != 0) {
      const uint4 v = aligned_load(s + 16, begin, end);
      w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
    }
    if (off & 8u) {
#pragma unroll
      for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    }
    if (off & 4u) {
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    }
    if (off & 2u) {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
    }
    const int64_t j = j0 + 8 * lane;
    if (j < a.cols)
      *reinterpret_cast<uint4*>(a.dst + i * a.ldd + j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 8 columns of dbias at a time, 32 runs of row blocks each.
__device__ __forceinline__ void add_dbias(const DbiasArgs& a) {
  __shared__ float part[32][9];
  const int r = threadIdx.x / 8, c = threadIdx.x % 8;
  for (int64_t j0 = static_cast<int64_t>(blockIdx.x) * 8; j0 < a.cols;
       j0 += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t j = j0 + c;
    float sum = 0.0f;
    if (j < a.cols) {
#pragma unroll 8
      for (int k = r; k < a.blocks; k += 32) sum += __ldcg(a.sums + k * round_up4(a.cols) + j);
    }
    __syncthreads();
    part[r][c] = sum;
    __syncthreads();
    if (r != 0 || j >= a.cols) continue;
#pragma unroll
    for (int k = 1; k < 32; ++k) sum += part[k][c];
    if (a.out_f32) {
      float* o = static_cast<float*>(a.dbias) + j;
      *o = a.accumulate ? *o + sum : sum;
    } else {
      uint16_t* o = static_cast<uint16_t*>(a.dbias) + j;
      *o = to_bf16(a.accumulate ? bf16_at(o) + sum : sum);
    }
  }
}

// Copies, a row of blocks each, or dbias (beside the products: it lets them begin).
__global__ void __launch_bounds__(256) linear_prepare_kernel(const __grid_constant__ PrepareArgs a) {
  wait_for_predecessor();
  launch_dependents();
  if (blockIdx.y < a.copies) copy_rows(a.copy[blockIdx.y]);
  else add_dbias(a.dbias);
}

// Takes pieces of the workspace in order.
struct Space {
  char* at;
  void* take(int64_t bytes) {
    void* p = at;
    at += round_up(bytes, 256);
    return p;
  }
};

// The kernels of one call, launched as programmatic dependents: they begin while
// their predecessor ends, and wait for it (wait_for_predecessor) before they read
// what it wrote; the first one so after whatever the stream held before.
struct Chain {
  cudaStream_t stream;
  bool begun = false;

  template <typename... Params, typename... Args>
  cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster,
                     Args&&... args) {
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    cudaLaunchAttribute attr[2];
    config.attrs = attr;
    if (cluster > 1) {
      cudaLaunchAttribute& a = attr[config.numAttrs++];
      a.id = cudaLaunchAttributeClusterDimension;
      a.val.clusterDim.x = cluster;
      a.val.clusterDim.y = 1;
      a.val.clusterDim.z = 1;
    }
    cudaLaunchAttribute& a = attr[config.numAttrs++];
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    begun = true;
    return cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...);
  }
};

// Lays the matrices that TMA cannot read where they are out anew.
cudaError_t lay_out(Stored* const* matrices, int count, Space* space, Chain* chain) {
  PrepareArgs all{};
  int64_t most = 0;
  for (int k = 0; k < count; ++k) {
    Stored& m = *matrices[k];
    if (m.p == nullptr || tileable(m)) continue;
    const int64_t pitch = copy_pitch(m.cols);
    CopyArgs& a = all.copy[all.copies++];
    a = {m.p, static_cast<uint16_t*>(space->take(copy_bytes(m))), m.rows, m.cols, m.ld, pitch};
    m.p = a.dst;
    m.ld = pitch;
    const int64_t blocks = (m.rows * ((m.cols + 255) / 256) + 7) / 8;
    most = blocks > most ? blocks : most;
  }
  if (all.copies == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(most < 2432 ? most : 2432), all.copies);
  return chain->launch(linear_prepare_kernel, grid, 256, 0, 1, all);
}

cudaError_t launch_dbias(const DbiasArgs& dbias, Chain* chain) {
  PrepareArgs all{};
  all.dbias = dbias;
  const int64_t blocks = (dbias.cols + 7) / 8;
  return chain->launch(linear_prepare_kernel, dim3(static_cast<unsigned>(blocks < 2432 ? blocks : 2432)),
                       256, 0, 1, all);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Boxes of 64 columns by `box_rows` rows, swizzled by 128 bytes; what lies past
// the matrix's edges reads as 0.
cudaError_t make_map(CUtensorMap* map, const Stored& m, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows)};
  const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(m.ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, unit[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(m.p), dims, pitch,
                box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// D or pre as `parts` matrices of rows x cols one after the other, in boxes of
// 32 x 32.
cudaError_t make_out_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld,
                         int64_t parts, int64_t stride, bool f32) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(parts)};
  const cuuint64_t pitch[2] = {static_cast<cuuint64_t>(ld * size),
                               static_cast<cuuint64_t>(stride * size)};
  const cuuint32_t box[3] = {32, 32, 1}, unit[3] = {1, 1, 1};
  return encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                const_cast<void*>(p), dims, pitch, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// ----------------------------------------------------------------- products

// D[rows, cols] over `depth`; a_mn / b_mn: the operand is stored [depth, rows]
// ([depth, cols]) instead of [rows, depth] ([cols, depth]).
struct Product {
  Stored a, b;
  bool a_mn, b_mn;
  int64_t rows, cols, depth;
  Epilogue e;
};

// A product under way: what its join needs, where its reduction is split.
struct Pending {
  ProductArgs a;
  Plan plan;
  int64_t rows;
  float* parts;
};

template <int CG, bool A_MN, bool B_MN, Kind KIND, bool ROWS, bool GATHER = false>
cudaError_t launch_shape(const Product& p, Pending* w, Chain* chain) {
  ProductArgs& a = w->a;
  const Plan& plan = w->plan;
  const int bn = plan.bn;
  auto kernel = linear_product_kernel<CG, A_MN, B_MN, KIND, ROWS, GATHER>;
  static std::mutex mu;
  static bool configured[64] = {false};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || device_sm_count(&sms) != 0) return cudaErrorNoDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  a.a_rows = a_rows_of(p.rows, CG, A_MN);
  e = make_map(&a.a, p.a, A_MN ? kDepth : a.a_rows);
  if (e == cudaSuccess) e = make_map(&a.b, p.b, B_MN ? kDepth : bn / CG);
  if (e != cudaSuccess) return e;
  const int64_t tm = (p.rows + CG * kBlockRows - 1) / (CG * kBlockRows), tn = (p.cols + bn - 1) / bn;
  if (tm * tn > INT32_MAX / 64) return cudaErrorInvalidValue;
  a.tiles_m = static_cast<int32_t>(tm);
  a.tiles_n = static_cast<int32_t>(tn);
  a.bn = bn;
  a.whole = plan.whole;
  a.splits = plan.splits;
  const int64_t units = grid_units(plan, sms);
  a.early_units = early_units_on(plan, units);
  a.early_tiles = plan.early_tiles;
  if (plan.splits > 1 && !GATHER) {
    e = make_out_map(&a.parts, w->parts, CG * kBlockRows, bn, bn, plan.tail * plan.splits,
                     CG * kBlockRows * bn, true);
    if (e != cudaSuccess) return e;
  }
  if (GATHER)  // a CTA for each item
    return chain->launch(kernel, dim3(static_cast<unsigned>(plan.tail * plan.splits)), kProductThreads,
                         kSmem, plan.splits, a);
  return chain->launch(kernel, dim3(static_cast<unsigned>(CG * units)), kProductThreads, kSmem, CG, a);
}

cudaError_t launch_join(const Pending& w, Chain* chain) {
  if (w.plan.splits == 1 || w.plan.gather) return cudaSuccess;
  const int64_t high = w.rows < w.plan.cg * kBlockRows ? w.rows : w.plan.cg * kBlockRows;
  const dim3 grid(static_cast<unsigned>((high * (w.plan.bn / 8) + 255) / 256), w.plan.tail);
  return w.plan.cg == 2 ? chain->launch(linear_join_kernel<256>, grid, 256, 0, 1, w.a, w.parts)
                        : chain->launch(linear_join_kernel<128>, grid, 256, 0, 1, w.a, w.parts);
}

template <bool A_MN, bool B_MN, Kind KIND>
cudaError_t launch_kind(const Product& p, Pending* w, Chain* chain) {
  if constexpr (!A_MN)
    if (w->plan.gather)
      return w->a.e.vec ? launch_shape<1, A_MN, B_MN, KIND, false, true>(p, w, chain)
                        : launch_shape<1, A_MN, B_MN, KIND, true, true>(p, w, chain);
  if constexpr (KIND != kFloat)
    if (!w->a.e.vec)
      return w->plan.cg == 2 ? launch_shape<2, A_MN, B_MN, KIND, true>(p, w, chain)
                             : launch_shape<1, A_MN, B_MN, KIND, true>(p, w, chain);
  return w->plan.cg == 2 ? launch_shape<2, A_MN, B_MN, KIND, false>(p, w, chain)
                         : launch_shape<1, A_MN, B_MN, KIND, false>(p, w, chain);
}

void set_vec(Epilogue* e, int64_t rows) {
  // (the pitch of a matrix of one row is not looked at)
  auto ok = [&](const void* p, int64_t ld, int bytes) {
    return p == nullptr || (aligned(p, 16) && (rows == 1 || ld * bytes % 16 == 0));
  };
  e->vec = ok(e->bias, 0, 2) && ok(e->pre, e->ldp, 2) && ok(e->residual, e->ldr, 2) &&
           ok(e->slope_of, e->lds, 2) && ok(e->out, e->ldo, e->out_f32 ? 4 : 2);
}

// late: see ProductArgs.  The join is left to the caller.
cudaError_t launch_product(Product p, const Plan& plan, bool late, Space* space, int withhold,
                           Chain* chain, Pending* w) {
  set_vec(&p.e, p.rows);
  *w = Pending{};
  w->plan = plan;
  w->rows = p.rows;
  w->parts = static_cast<float*>(space->take(plan.part_bytes()));
  ProductArgs& a = w->a;
  a.e = p.e;
  a.rows = p.rows;
  a.cols = p.cols;
  a.steps = static_cast<int32_t>((p.depth + kStep - 1) / kStep);
  a.withhold = withhold;
  a.late = late;
  const bool f32 = a.e.out_f32 != 0;
  if (a.e.vec) {
    // a matrix of one row has any pitch
    const int64_t one = round_up(p.cols, 8);
    const int64_t stride = p.rows > 1 ? p.rows * a.e.ldo : one;
    cudaError_t e =
        make_out_map(&a.out, a.e.out, p.rows, p.cols, p.rows > 1 ? a.e.ldo : one, 1, stride, f32);
    if (e == cudaSuccess && a.e.pre != nullptr)
      e = make_out_map(&a.pre, a.e.pre, p.rows, p.cols, p.rows > 1 ? a.e.ldp : one, 1, stride, false);
    if (e != cudaSuccess) return e;
  }
  if (p.a_mn)
    return f32 ? launch_kind<true, true, kFloat>(p, w, chain)
               : launch_kind<true, true, kGradient>(p, w, chain);
  if (p.b_mn) return launch_kind<false, true, kGradient>(p, w, chain);
  return launch_kind<false, false, kForward>(p, w, chain);
}

// --------------------------------------------------------------- a few rows
//
// y for at most 16 rows of x (tokens of generation): W is read once and nothing
// else counts, so this is bound by HBM bandwidth.  A warp takes 16 rows of W, a
// block's 8 warps share out the columns, and the warp-level matrix instruction
// (16 rows of W by 8 rows of x, 16 steps) adds up.  4096 x 11008, calls in a row
// over cold weights: 1 row 16.2 us (5.6 TB/s; fp32 multiply-adds instead of
// matrix instructions were level there and 7 times slower at 8), 8 rows 17.8, 16
// rows 21.2; tcgen05's tiles, brought through shared memory, 21.3 for any number
// up to 32, so they take over at 17.  A lane's 16-byte load is 8 neighbours of one row; which steps of
// the reduction an instruction's operands belong to does not matter as long as
// W's and x's agree, so the vectors are its operands as they are.  All loads of
// 64 or 128 columns are in flight at once; x comes from L1.  The shares are
// added through shared memory in their order.

constexpr int kFewRows = 16, kFewWarps = 8;

struct FewArgs {
  const uint16_t *x, *w;
  int64_t ldx, ldw;
  int64_t cols;   // of D: rows of W
  int32_t depth, rows;
  int32_t share;  // warps that share out the columns of 16 rows of W: 1, 2, 4 or 8
  Epilogue e;
};

// 8 elements from p[j] on; those from n on are 0.  (Columns are counted without a
// sign: n may be 2^31 - 2, and a warp's place passes it by up to a round of the block.)
template <bool VEC, bool STREAM>
__device__ __forceinline__ uint4 few_load(const uint16_t* p, uint32_t j, uint32_t n) {
  if (VEC && j + 8 <= n) {
    uint4 v;
    if (STREAM)
      asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(p + j));
    else
      v = __ldg(reinterpret_cast<const uint4*>(p + j));
    return v;
  }
  uint32_t w[4] = {};
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (j + c < n) w[c / 2] |= static_cast<uint32_t>(__ldg(p + j + c)) << (16 * (c & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// d += the product of 16 rows (a) and 8 rows (b) over 16 steps.
__device__ __forceinline__ void warp_mma(float d[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 rows of x; U: loads of each row in flight.
template <int NT, int U, bool VEC>
__global__ void __launch_bounds__(32 * kFewWarps, U == 2 ? 5 : 3)
    linear_few_rows_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kSpan = 32 * U;          // columns a warp takes at a time
  __shared__ float part[kFewWarps][16 * 8 * NT];
  wait_for_predecessor();
  launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int share = a.share, mine = warp % share;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * (kFewWarps / share) + warp / share) * 16;
  float acc[NT][4] = {};
  if (row0 < a.cols) {
    // rows past the end read the last one; nothing is made of them
    const int64_t top = row0 + g, low = row0 + g + 8, end = a.cols - 1;
    const uint16_t* w0 = a.w + (top < end ? top : end) * a.ldw;
    const uint16_t* w1 = a.w + (low < end ? low : end) * a.ldw;
    const uint16_t* x[NT];  // rows past the end: row 0's, in sums that are not stored
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = a.x + (8 * n + g < a.rows ? 8 * n + g : 0) * a.ldx;
    const uint32_t depth = a.depth;
    for (uint32_t k0 = kSpan * mine; k0 < depth; k0 += kSpan * share) {
      const uint32_t j = k0 + 8 * t;
      uint4 u[U], v[U];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        u[q] = few_load<VEC, true>(w0, j + 32 * q, depth);
        v[q] = few_load<VEC, true>(w1, j + 32 * q, depth);
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 y = few_load<VEC, false>(x[n], j + 32 * q, depth);
          warp_mma(acc[n], u[q].x, v[q].x, u[q].y, v[q].y, y.x, y.y);
          warp_mma(acc[n], u[q].z, v[q].z, u[q].w, v[q].w, y.z, y.w);
        }
      }
    }
  }
  // (row of W, row of x) of a lane's sums: (g, 2t), (g, 2t + 1), and g + 8 alike
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      part[warp][(8 * n + 2 * t + c % 2) * 16 + g + 8 * (c / 2)] = acc[n][c];
  __syncthreads();
  // one thread an output, neighbours along W's rows
  for (int q = threadIdx.x; q < (kFewWarps / share) * 128 * NT; q += 32 * kFewWarps) {
    const int group = q / (128 * NT), in = q % (128 * NT), m = in / 16;
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * (kFewWarps / share) + group) * 16 + in % 16;
    if (j >= a.cols || m >= a.rows) continue;
    float sum = 0.0f;
    for (int s = 0; s < share; ++s) sum += part[group * share + s][in];
    epilogue_element(a.e, m, j, sum);
  }
}

template <int NT>
cudaError_t launch_few_groups(FewArgs& a, bool vec, Chain* chain) {
  // The columns are shared out until there are 16 warps an SM, or a warp's part
  // is one step.
  const int64_t groups = (a.cols + 15) / 16;
  a.share = 1;
  while (a.share < kFewWarps && groups * a.share < int64_t{32} * kSms && a.depth > 128 * a.share)
    a.share *= 2;
  const int64_t blocks = (groups + kFewWarps / a.share - 1) / (kFewWarps / a.share);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  // Many blocks: few registers, 5 blocks an SM; few: more in flight by each warp
  // (1 x 4096 x 11008, 688 blocks: 16.2 us against 19.5 with the 4 loads that 1 x
  // 11008 x 4096, 256 blocks, wants: 18.5 against 25.1).
  const unsigned grid = static_cast<unsigned>(blocks), threads = 32 * kFewWarps;
  const auto kernel = blocks >= 3 * kSms ? (vec ? linear_few_rows_kernel<NT, 2, true>
                                                : linear_few_rows_kernel<NT, 2, false>)
                                         : (vec ? linear_few_rows_kernel<NT, 4, true>
                                                : linear_few_rows_kernel<NT, 4, false>);
  return chain->launch(kernel, dim3(grid), threads, 0, 1, a);
}
cudaError_t launch_few_rows(const Product& p, Chain* chain) {
  FewArgs a{};
  a.x = p.a.p;
  a.ldx = p.a.ld;
  a.w = p.b.p;
  a.ldw = p.b.ld;
  a.rows = static_cast<int32_t>(p.rows);
  a.cols = p.cols;
  a.depth = static_cast<int32_t>(p.depth);
  a.e = p.e;
  const bool vec = tileable(p.a) && tileable(p.b);
  return p.rows <= 8 ? launch_few_groups<1>(a, vec, chain) : launch_few_groups<2>(a, vec, chain);
}

// dz = bf16(dy * act'(pre)), and each column's sum of it before the rounding.
// The products take dz as bf16, as the tensor cores' operands are: with x or W exact
// that puts dx and dw 0.0023 from the exact ones in the 2-norm where their own
// rounding puts them 0.0017; carrying the remainder in a second product would double
// both products' time.
// One pass over dy and pre, bound by HBM bandwidth.  A warp takes 256 columns of
// every row of its block's, 8 a lane, and the block's 4 warps lie side by side, so
// that a row is read 2 KB at a time; its column sums, a thread's own, go to the
// workspace, and add_dbias adds the blocks' in their order.
constexpr int kSlopeWarps = 4, kSlopeCols = 256 * kSlopeWarps;

struct SlopeArgs {
  const uint16_t *dy, *pre;
  int64_t ldy, ldp, rows, cols;
  int32_t vec;     // 16-byte accesses
  int32_t height;  // rows of a block
  uint16_t* dz;    // NULL: sums only
  int64_t ldz;
  float* sums;     // [row blocks][cols], NULL: dz only
  int32_t late;    // as in ProductArgs
};

template <int ACT>
__device__ __forceinline__ void slope_rows(const SlopeArgs& a, int64_t j0, int lane) {
  const int64_t first = static_cast<int64_t>(blockIdx.y) * a.height;
  const int n = static_cast<int>(a.rows - first < a.height ? a.rows - first : a.height);
  float sum[8] = {};
  if (a.vec && j0 + 256 <= a.cols) {
    const int64_t j = j0 + 8 * lane;
    const uint16_t* dy = a.dy + first * a.ldy + j;
    const uint16_t* pre = ACT != ZERO_ACT_NONE ? a.pre + first * a.ldp + j : dy;
    uint16_t* dz = a.dz != nullptr ? a.dz + first * a.ldz + j : nullptr;
    // 4 rows' loads at a time: one row's are too few to cover HBM's latency
#pragma unroll 1
    for (int i = 0; i < n; i += 4) {
      uint4 u[4], w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i + k >= n) break;
        u[k] = __ldcs(reinterpret_cast<const uint4*>(dy + k * a.ldy));
        if (ACT != ZERO_ACT_NONE) w[k] = __ldcs(reinterpret_cast<const uint4*>(pre + k * a.ldp));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i + k >= n) break;
        float x[8];
        bf16x8(u[k], x);
        if (ACT != ZERO_ACT_NONE) times_slope8(x, w[k], ACT);
        if (dz != nullptr) *reinterpret_cast<uint4*>(dz + k * a.ldz) = to_bf16x8(x);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += x[c];
      }
      dy += 4 * a.ldy;
      pre += 4 * a.ldp;
      if (dz != nullptr) dz += 4 * a.ldz;
    }
    if (a.sums != nullptr) {
      float4* s = reinterpret_cast<float4*>(a.sums + blockIdx.y * round_up4(a.cols) + j);
      s[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
      s[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < n; i += 2) {  // 2 rows' loads at a time
      float x[2][8], z[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int64_t j = j0 + 32 * c + lane;
          const bool in = j < a.cols && i + k < n;
          x[k][c] = in ? bf16_at(a.dy + (first + i + k) * a.ldy + j) : 0.0f;
          if (ACT != ZERO_ACT_NONE) z[k][c] = in ? bf16_at(a.pre + (first + i + k) * a.ldp + j) : 0.0f;
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int64_t j = j0 + 32 * c + lane;
          if (ACT != ZERO_ACT_NONE && c % 2 == 0)
            times_slope2<ACT>(x[k][c], x[k][c + 1], z[k][c], z[k][c + 1]);
          if (a.dz != nullptr && j < a.cols && i + k < n)
            a.dz[(first + i + k) * a.ldz + j] = to_bf16(x[k][c]);
          sum[c] += x[k][c];
        }
    }
    if (a.sums != nullptr) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int64_t j = j0 + 32 * c + lane;
        if (j < a.cols) a.sums[blockIdx.y * round_up4(a.cols) + j] = sum[c];
      }
    }
  }
}

template <int ACT>
__global__ void __launch_bounds__(32 * kSlopeWarps, 6)
    linear_slope_kernel(const __grid_constant__ SlopeArgs a) {
  if (!a.late) wait_for_predecessor();
  launch_dependents();
  const int64_t j0 =
      static_cast<int64_t>(blockIdx.x) * kSlopeCols + 256 * static_cast<int>(threadIdx.x / 32);
  if (j0 < a.cols) slope_rows<ACT>(a, j0, threadIdx.x % 32);
  if (a.late) wait_for_predecessor();
}

// Rows of a block: 8 blocks an SM, 4 to 64 rows.
int64_t slope_height(int64_t rows, int64_t cols) {
  const int64_t across = (cols + kSlopeCols - 1) / kSlopeCols;
  const int64_t h = rows * across / (8 * kSms);
  return h < 4 ? 4 : h > 64 ? 64 : h;
}
int64_t slope_blocks(int64_t rows, int64_t cols) {
  const int64_t h = slope_height(rows, cols);
  return (rows + h - 1) / h;
}

}  // namespace

int read_and_clear_linear_status(int* status) {
  take_linear_status_kernel<<<1, 1, 0, 0>>>();
  if (cudaGetLastError() != cudaSuccess) return -1;
  int v = 0;  // the copy is ordered after the kernel on the legacy default stream
  if (cudaMemcpyFromSymbol(&v, g_linear_status_taken, sizeof(int)) != cudaSuccess) return -1;
  *status = v;
  return 0;
}

int64_t linear_workspace(const zero_linear_t& s, int32_t flags) {
  const bool in_place = (flags & ZERO_LINEAR_ALIGNED) != 0;
  const int64_t x = in_place ? 0 : copy_bytes(Stored(nullptr, s.rows, s.in, 0));
  const int64_t w = in_place ? 0 : copy_bytes(Stored(nullptr, s.out, s.in, 0));
  const int64_t bias = in_place ? 0 : copy_bytes(Stored(nullptr, 1, s.out, 0));
  if ((flags & ZERO_LINEAR_BACKWARD) == 0)
    return s.rows <= kFewRows ? 0 : x + w + bias + round_up(plan_forward(s).part_bytes(), 256);
  const bool dz = !in_place || (flags & ZERO_LINEAR_PLAIN) == 0;
  // the two products' parts, side by side; either may be wanted alone
  const BackwardPlan both = plan_backward(s, true, true), one = plan_backward(s, true, false),
                     two = plan_backward(s, false, true);
  auto most = [](int64_t x, int64_t y) { return x > y ? x : y; };
  return (dz ? copy_bytes(Stored(nullptr, s.rows, s.out, 0)) : 0) + w + x +
         round_up(slope_blocks(s.rows, s.out) * round_up4(s.out) * 4, 256) +
         most(both.dx.part_bytes() + both.dw.part_bytes(),
              most(one.dx.part_bytes(), two.dw.part_bytes())) + 512;
}

cudaError_t launch_linear_forward(const LinearForwardLaunch& L) {
  (void)cudaGetLastError();
  const zero_linear_t& s = L.s;
  Product p{};
  p.a = {L.x, s.rows, s.in, s.ldx};
  p.b = {L.w, s.out, s.in, s.ldw};
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
  Chain chain{L.stream};
  if (s.rows <= kFewRows) return launch_few_rows(p, &chain);
  Space space{static_cast<char*>(L.workspace)};
  // (where only the bias is out of place, its copy costs a launch; taken element by
  // element it would take the whole epilogue with it)
  Stored bias{L.bias, 1, s.out, 0};
  Stored* const all[3] = {&p.a, &p.b, &bias};
  cudaError_t e = lay_out(all, 3, &space, &chain);
  p.e.bias = bias.p;
  Pending w;
  if (e == cudaSuccess)
    e = launch_product(p, plan_forward(s), false, &space, L.withhold, &chain, &w);
  return e == cudaSuccess ? launch_join(w, &chain) : e;
}

cudaError_t launch_linear_backward(const LinearBackwardLaunch& L) {
  (void)cudaGetLastError();
  const zero_linear_t& s = L.s;
  Stored dz{L.dy, s.rows, s.out, s.ldy};
  Space space{static_cast<char*>(L.workspace)};
  Chain chain{L.stream};
  DbiasArgs dbias{};
  dbias.cols = s.out;
  dbias.dbias = L.dbias;
  dbias.out_f32 = L.grad_f32;
  dbias.accumulate = L.accumulate;
  if (s.rows == 0) {  // sums of nothing
    const cudaError_t e = L.dbias != nullptr ? launch_dbias(dbias, &chain) : cudaSuccess;
    if (e != cudaSuccess || L.dw == nullptr || L.accumulate) return e;
    return cudaMemset2DAsync(L.dw, s.lddw * (L.grad_f32 ? 4 : 2), 0, s.in * (L.grad_f32 ? 4 : 2),
                             s.out, L.stream);
  }
  const bool products = L.dx != nullptr || L.dw != nullptr;
  SlopeArgs a{};
  if (L.act != ZERO_ACT_NONE && products) {
    a.dz = static_cast<uint16_t*>(space.take(copy_bytes(dz)));
    a.ldz = copy_pitch(s.out);
    dz = Stored(a.dz, s.rows, s.out, a.ldz);
  }
  if (!products) dz.p = nullptr;
  Stored w(L.dx != nullptr ? L.w : nullptr, s.out, s.in, s.ldw);
  Stored x(L.dw != nullptr ? L.x : nullptr, s.rows, s.in, s.ldx);
  Stored* const all[3] = {&dz, &w, &x};
  cudaError_t e = lay_out(all, 3, &space, &chain);
  if (e != cudaSuccess) return e;
  if (a.dz != nullptr || L.dbias != nullptr) {
    a.dy = L.dy;
    a.pre = L.pre;
    a.ldy = s.ldy;
    a.ldp = s.ldp;
    a.rows = s.rows;
    a.cols = s.out;
    const int64_t blocks = slope_blocks(s.rows, s.out);
    a.height = static_cast<int32_t>(slope_height(s.rows, s.out));
    if (L.dbias != nullptr) {
      a.sums = static_cast<float*>(space.take(blocks * round_up4(s.out) * 4));
      dbias.sums = a.sums;
      dbias.blocks = static_cast<int32_t>(blocks);
    }
    a.vec = tileable(Stored(L.dy, s.rows, s.out, s.ldy)) &&
            (L.act == ZERO_ACT_NONE || tileable(Stored(L.pre, s.rows, s.out, s.ldp)));
    a.late = chain.begun;  // beside the copies
    auto kernel = L.act == ZERO_ACT_GELU   ? linear_slope_kernel<ZERO_ACT_GELU>
                  : L.act == ZERO_ACT_SILU ? linear_slope_kernel<ZERO_ACT_SILU>
                  : L.act == ZERO_ACT_RELU ? linear_slope_kernel<ZERO_ACT_RELU>
                                           : linear_slope_kernel<ZERO_ACT_NONE>;
    const int64_t across = (s.out + kSlopeCols - 1) / kSlopeCols;
    // the grid's y side ends at 65535
    for (int64_t k = 0; k < blocks && e == cudaSuccess; k += 65535) {
      SlopeArgs part = a;
      const int64_t skip = k * a.height;
      part.dy += skip * s.ldy;
      part.pre += L.act != ZERO_ACT_NONE ? skip * s.ldp : 0;
      part.dz += a.dz != nullptr ? skip * a.ldz : 0;
      part.sums += a.sums != nullptr ? k * round_up4(s.out) : 0;
      part.rows -= skip;
      part.late = a.late && k == 0;
      const int64_t high = blocks - k < 65535 ? blocks - k : 65535;
      const dim3 grid(static_cast<unsigned>(across), static_cast<unsigned>(high));
      e = chain.launch(kernel, grid, 32 * kSlopeWarps, 0, 1, part);
    }
    if (e == cudaSuccess && L.dbias != nullptr) e = launch_dbias(dbias, &chain);
    if (e != cudaSuccess) return e;
  }
  const BackwardPlan plan = plan_backward(s, L.dx != nullptr, L.dw != nullptr);
  Pending dx{}, dw{};
  dx.plan.splits = dw.plan.splits = 1;
  if (L.dx != nullptr) {
    Product p{};
    p.a = dz;
    p.b = w;
    p.b_mn = true;
    p.rows = s.rows;
    p.cols = s.in;
    p.depth = s.out;
    p.e.slope_act = L.act_in;
    p.e.slope_of = L.act_in != ZERO_ACT_NONE ? L.pre_in : nullptr;
    p.e.lds = s.ldpi;
    p.e.out = L.dx;
    p.e.ldo = s.lddx;
    // dbias's kernel has waited for all that this one reads before it let it begin
    e = launch_product(p, plan.dx, L.dbias != nullptr, &space, L.withhold, &chain, &dx);
    if (e != cudaSuccess) return e;
  }
  if (L.dw != nullptr) {
    Product p{};
    p.a = dz;
    p.a_mn = true;
    p.b = x;
    p.b_mn = true;
    p.rows = s.out;
    p.cols = s.in;
    p.depth = s.rows;
    p.e.out = L.dw;
    p.e.ldo = s.lddw;
    p.e.out_f32 = L.grad_f32;
    p.e.accumulate = L.accumulate;
    // (and so have dx's product, or what came before that)
    e = launch_product(p, plan.dw, L.dbias != nullptr || L.dx != nullptr, &space, L.withhold, &chain, &dw);
    if (e != cudaSuccess) return e;
  }
  e = launch_join(dx, &chain);
  return e == cudaSuccess ? launch_join(dw, &chain) : e;
}

}  // namespace zeroadam
