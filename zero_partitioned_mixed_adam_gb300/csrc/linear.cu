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

#include "internal.h"
#include "linear_epilogue.cuh"
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

constexpr int kDepth = 64;         // steps of the reduction in one stage: 128 bytes of bf16
constexpr int kBlockRows = 128;    // rows of D per CTA: the lanes of tensor memory
constexpr int kEpilogueWarps = 8;  // two per quarter of the lanes
constexpr int kProductThreads = 64 + 32 * kEpilogueWarps;

// One tile of D is CG * 128 rows by BN columns, made by CG CTAs: each brings
// its own 128 rows of A and BN/CG rows of B, the tensor cores read both CTAs'
// B (half the shared-memory traffic of two tiles of their own), and each CTA's
// tensor memory ends up with its 128 rows.
template <int CG, int BN>
struct ProductShape {
  static constexpr int kBRows = BN / CG;
  static constexpr int kABytes = kBlockRows * kDepth * 2;
  static constexpr int kBBytes = kBRows * kDepth * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStaging = kEpilogueWarps * 32 * 32 * 4;
  static constexpr int kBarriers = 512;
  static constexpr int kStages = (227 * 1024 - 1024 - kStaging - kBarriers) / kStage;
  static constexpr int kSmem = kStages * kStage + kStaging + kBarriers + 1024;
  static constexpr int kColumns = 2 * BN < 32 ? 32 : 2 * BN;  // of tensor memory: two tiles
  static_assert(kStages >= 3 && 2 * kStages + 5 <= kBarriers / 8, "stages");
  static_assert(kColumns <= 512 && BN % 64 == 0, "tensor memory");
};

struct ProductArgs {
  CUtensorMap a, b;
  Epilogue e;
  int64_t rows, cols;
  int64_t split_stride;  // elements of D between two parts of a split reduction
  int32_t tiles_m, tiles_n, splits;
  int32_t steps;         // stages of the whole reduction
  int32_t withhold;      // test hook: no loads are issued, so every wait runs out
};

struct Tile {
  int64_t row, col;   // of the tile's first element
  int first, last;    // stages
  int split;
};

// Tiles in the order CTAs take them: the parts of the reduction apart, and in
// each part columns of up to 8 tiles of rows, so that the tiles in flight at
// one time share their operands in L2.
template <int BM, int BN>
__device__ __forceinline__ Tile tile_of(const ProductArgs& a, int t) {
  constexpr int kGroup = 8;
  const int per = a.tiles_m * a.tiles_n;
  Tile r;
  r.split = t / per;
  t -= r.split * per;
  const int group = t / (kGroup * a.tiles_n);
  const int m0 = group * kGroup;
  const int height = a.tiles_m - m0 < kGroup ? a.tiles_m - m0 : kGroup;
  const int in = t - group * kGroup * a.tiles_n;
  r.row = static_cast<int64_t>(m0 + in % height) * BM;
  r.col = static_cast<int64_t>(in / height) * BN;
  r.first = static_cast<int>(static_cast<int64_t>(a.steps) * r.split / a.splits);
  r.last = static_cast<int>(static_cast<int64_t>(a.steps) * (r.split + 1) / a.splits);
  return r;
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
template <int CG, int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kProductThreads, 1)
    linear_product_kernel(const __grid_constant__ ProductArgs a) {
  using Shape = ProductShape<CG, BN>;
  constexpr int kStages = Shape::kStages;
  constexpr int BM = CG * kBlockRows;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  float* staging = reinterpret_cast<float*>(ring + kStages * Shape::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * Shape::kStage + Shape::kStaging);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint64_t* free_ = done + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(free_ + 2);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int unit = blockIdx.x / CG, units = gridDim.x / CG;
  const int tiles = a.tiles_m * a.tiles_n * a.splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&done[b], 1);
      mbar_init(&free_[b], kEpilogueWarps * CG);
    }
    mbar_init_fence();
    prefetch_map(&a.a);
    prefetch_map(&a.b);
  }
  if (warp == 1) tmem_alloc<CG>(tmem_at, Shape::kColumns);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp == 0) {
    if (lane == 0) {
      int64_t k = 0;  // stages issued
      bool ok = true;
      for (int t = unit; t < tiles && ok; t += units) {
        const Tile tile = tile_of<BM, BN>(a, t);
        const int ra = static_cast<int>(tile.row) + rank * kBlockRows;
        const int rb = static_cast<int>(tile.col) + rank * Shape::kBRows;
        for (int step = tile.first; step < tile.last; ++step, ++k) {
          const int s = static_cast<int>(k % kStages);
          if (k >= kStages && !mbar_wait(&empty[s], static_cast<uint32_t>((k / kStages - 1) & 1))) {
            ok = false;
            break;
          }
          if (a.withhold) continue;
          uint8_t* sa = ring + s * Shape::kStage;
          uint8_t* sb = sa + Shape::kABytes;
          const uint32_t bar = CG == 2 ? peer_addr(&full[s], 0) : smem_addr(&full[s]);
          if (rank == 0) mbar_expect_tx(&full[s], CG * Shape::kStage);
          const int x = step * kDepth;
          if constexpr (A_MN) {
#pragma unroll
            for (int c = 0; c < kBlockRows / 64; ++c)
              tile_load<CG>(sa + c * 64 * kDepth * 2, &a.a, ra + 64 * c, x, bar);
          } else {
            tile_load<CG>(sa, &a.a, x, ra, bar);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int c = 0; c < Shape::kBRows / 64; ++c)
              tile_load<CG>(sb + c * 64 * kDepth * 2, &a.b, rb + 64 * c, x, bar);
          } else {
            tile_load<CG>(sb, &a.b, x, rb, bar);
          }
        }
      }
      if (!ok) atomicExch(&g_linear_status, 1);
      // No CTA ends while loads into it, or arrivals on its barriers, are under
      // way: the products that read the last stages are waited for.
      if (!a.withhold)
        for (int64_t j = k > kStages ? k - kStages : 0; j < k; ++j)
          mbar_wait(&empty[j % kStages], static_cast<uint32_t>((j / kStages) & 1));
      if (!ok && rank == 0 && !a.withhold)
        for (int64_t j = k > kStages ? k - kStages : 0; j < k; ++j)
          mbar_wait(&full[j % kStages], static_cast<uint32_t>((j / kStages) & 1));
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t desc = mma_desc(BM, BN, A_MN, B_MN);
      // bytes between two steps of 16 of the reduction, and the distances of
      // smem_desc, along each operand's rows
      constexpr uint32_t step_a = A_MN ? 16 * 128 : 32, step_b = B_MN ? 16 * 128 : 32;
      constexpr uint32_t lead = 64 * kDepth * 2, stride = 1024;
      int64_t k = 0;
      int n = 0;  // tiles begun
      bool ok = true;
      for (int t = unit; t < tiles && ok; t += units, ++n) {
        const Tile tile = tile_of<BM, BN>(a, t);
        const int b = n & 1;
        if (n >= 2 && !mbar_wait(&free_[b], static_cast<uint32_t>((n / 2 - 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int step = tile.first; step < tile.last; ++step, ++k) {
          const int s = static_cast<int>(k % kStages);
          if (!mbar_wait(&full[s], static_cast<uint32_t>((k / kStages) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_addr(ring + s * Shape::kStage), sb = sa + Shape::kABytes;
          const uint64_t da = smem_desc(sa, lead, stride), db = smem_desc(sb, lead, stride);
#pragma unroll
          for (int q = 0; q < kDepth / 16; ++q)
            mma_bf16<CG>(tmem + b * BN, da + q * (step_a >> 4), db + q * (step_b >> 4), desc,
                         step > tile.first || q > 0);
          mma_commit<CG>(&empty[s]);
        }
        if (ok) mma_commit<CG>(&done[b]);
      }
      if (!ok) {
        // products already issued end before tensor memory is freed
        atomicExch(&g_linear_status, 2);
        for (int64_t j = k > kStages ? k - kStages : 0; j < k; ++j)
          mbar_wait(&empty[j % kStages], static_cast<uint32_t>((j / kStages) & 1));
      }
    }
  } else {
    const int quarter = warp % 4, half = (warp - 2) / 4;
    float* mine = staging + (warp - 2) * 32 * 32;
    int n = 0;
    for (int t = unit; t < tiles; t += units, ++n) {
      const Tile tile = tile_of<BM, BN>(a, t);
      const int b = n & 1;
      if (!mbar_wait(&done[b], static_cast<uint32_t>((n / 2) & 1))) {
        if (lane == 0) atomicExch(&g_linear_status, 3);
        break;
      }
      tc_fence_after();
      const int64_t row0 = tile.row + rank * kBlockRows + quarter * 32;
      Epilogue e = a.e;
      e.out = e.out_f32 ? static_cast<void*>(static_cast<float*>(e.out) + tile.split * a.split_stride)
                        : e.out;
#pragma unroll 1
      for (int c = 0; c < BN / 2; c += 32) {
        const int at = half * (BN / 2) + c;
        uint32_t x[32];
        tmem_load32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * BN + at, x);
        tmem_load_wait();
        if (c + 32 >= BN / 2) {  // the warp has read its part: this half may be written again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_peer(peer_addr(&free_[b], 0));
            else mbar_arrive(&free_[b]);
          }
        }
        // Through shared memory into rows: a lane holds 32 columns of one row, and
        // takes 4 columns of 8 rows, so that 8 lanes cover a row's 32.  The 16-byte
        // pieces of a row are permuted by its number, against bank conflicts.
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(mine + lane * 32 + ((q ^ (lane & 7)) * 4)) =
              make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        __syncwarp();
        const int64_t j = tile.col + at + 4 * (lane % 8);
        const int cols = a.cols - j < 4 ? (a.cols > j ? static_cast<int>(a.cols - j) : 0) : 4;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          EpilogueInputs in[4];
          float d[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = (4 * g + q) * 4 + lane / 8;
            const float4 v = *reinterpret_cast<const float4*>(
                mine + r * 32 + (((lane % 8) ^ (r & 7)) * 4));
            d[q][0] = v.x; d[q][1] = v.y; d[q][2] = v.z; d[q][3] = v.w;
            if (cols > 0 && row0 + r < a.rows) epilogue_load4(e, row0 + r, j, cols, in[q]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = (4 * g + q) * 4 + lane / 8;
            if (cols > 0 && row0 + r < a.rows) epilogue_store4(e, row0 + r, j, cols, in[q], d[q]);
          }
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) tmem_free<CG>(tmem, Shape::kColumns);
}

// The parts of a split reduction, added in their order, and the epilogue.
struct JoinArgs {
  const float* parts;
  int64_t ld, stride;
  int32_t splits;
  int64_t rows, cols;
  Epilogue e;
};

__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ JoinArgs a) {
  const int64_t quads = (a.cols + 3) / 4;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < a.rows * quads;
       q += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t i = q / quads, j = (q - i * quads) * 4;
    const int n = a.cols - j < 4 ? static_cast<int>(a.cols - j) : 4;
    EpilogueInputs in;
    epilogue_load4(a.e, i, j, n, in);
    float x[4] = {};
    for (int s = 0; s < a.splits; ++s) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.parts + s * a.stride + i * a.ld + j));
      x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w;
    }
    epilogue_store4(a.e, i, j, n, in, x);
  }
}

// ------------------------------------------------------------------ layouts

int64_t round_up(int64_t x, int64_t k) { return (x + k - 1) / k * k; }
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
int64_t copy_bytes(const Stored& m) { return round_up(m.rows * round_up(m.cols, 8) * 2, 256); }

struct CopyArgs {
  const uint16_t* src;
  uint16_t* dst;
  int64_t rows, cols, lds, ldd;
};

// A matrix laid out anew with rows on 16-byte boundaries: 8 elements a thread.
__global__ void __launch_bounds__(256) linear_copy_kernel(const __grid_constant__ CopyArgs a) {
  const int64_t per = (a.cols + 7) / 8;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; q < a.rows * per;
       q += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t i = q / per, j = (q - i * per) * 8;
    const uint16_t* s = a.src + i * a.lds + j;
    uint32_t w[4] = {};
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (j + c < a.cols) w[c / 2] |= static_cast<uint32_t>(__ldg(s + c)) << (16 * (c & 1));
    *reinterpret_cast<uint4*>(a.dst + i * a.ldd + j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
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

cudaError_t make_tileable(Stored* m, Space* space, cudaStream_t stream) {
  if (tileable(*m)) return cudaSuccess;
  CopyArgs a{m->p, static_cast<uint16_t*>(space->take(copy_bytes(*m))), m->rows, m->cols, m->ld,
             round_up(m->cols, 8)};
  const int64_t blocks = (m->rows * (a.ldd / 8) + 255) / 256;
  linear_copy_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(a);
  m->p = a.dst;
  m->ld = a.ldd;
  return cudaGetLastError();
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

// ----------------------------------------------------------------- products

// D[rows, cols] over `depth`; a_mn / b_mn: the operand is stored [depth, rows]
// ([depth, cols]) instead of [rows, depth] ([cols, depth]).
struct Product {
  Stored a, b;
  bool a_mn, b_mn;
  int64_t rows, cols, depth;
  Epilogue e;
};

// Planned for the part's 152 SMs wherever it runs, so that the sums' order and
// the workspace follow from the sizes alone.
constexpr int kSms = 152;

struct Plan {
  int cg, bn, splits;
};

Plan plan_product(int64_t rows, int64_t cols, int64_t depth) {
  const int64_t steps = (depth + kDepth - 1) / kDepth;
  Plan best{2, 256, 1};
  if (rows < 1 || cols < 1) return best;
  double least = 1e300;
  const struct { int cg, bn; double rate; } shapes[] = {{2, 256, 1.0}, {2, 128, 0.85}, {1, 128, 0.7}};
  for (const auto& s : shapes) {
    const int64_t tiles = ((rows + 128 * s.cg - 1) / (128 * s.cg)) * ((cols + s.bn - 1) / s.bn);
    const int64_t units = kSms / s.cg;
    const int64_t waves = (tiles + units - 1) / units;
    const double cost = waves * (128.0 * s.bn) / s.rate;
    if (cost < least) {
      least = cost;
      best.cg = s.cg;
      best.bn = s.bn;
      int64_t splits = 1;
      if (tiles * 2 <= units) {  // most SMs would idle: the reduction is cut
        splits = units / tiles;
        if (splits > steps / 4) splits = steps / 4;
        if (splits > 16) splits = 16;
        if (splits < 1) splits = 1;
      }
      best.splits = static_cast<int>(splits);
    }
  }
  return best;
}

int64_t parts_bytes(const Plan& p, int64_t rows, int64_t cols) {
  return p.splits > 1 ? round_up(p.splits * rows * round_up(cols, 4) * 4, 256) : 0;
}

template <int CG, int BN, bool A_MN, bool B_MN>
cudaError_t launch_shape(const Product& p, const Plan& plan, ProductArgs& a, cudaStream_t stream) {
  using Shape = ProductShape<CG, BN>;
  auto kernel = linear_product_kernel<CG, BN, A_MN, B_MN>;
  static std::mutex mu;
  static bool configured[64] = {false};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || device_sm_count(&sms) != 0) return cudaErrorNoDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  e = make_map(&a.a, p.a, A_MN ? kDepth : kBlockRows);
  if (e == cudaSuccess) e = make_map(&a.b, p.b, B_MN ? kDepth : Shape::kBRows);
  if (e != cudaSuccess) return e;
  const int64_t tm = (p.rows + CG * kBlockRows - 1) / (CG * kBlockRows), tn = (p.cols + BN - 1) / BN;
  if (tm * tn * plan.splits > INT32_MAX) return cudaErrorInvalidValue;
  a.tiles_m = static_cast<int32_t>(tm);
  a.tiles_n = static_cast<int32_t>(tn);
  const int64_t units = sms / CG, tiles = tm * tn * plan.splits;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(static_cast<unsigned>(CG * (tiles < units ? tiles : units)));
  config.blockDim = dim3(kProductThreads);
  config.dynamicSmemBytes = Shape::kSmem;
  config.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  config.attrs = attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, a);
}

template <bool A_MN, bool B_MN>
cudaError_t launch_majors(const Product& p, const Plan& plan, ProductArgs& a, cudaStream_t stream) {
  if (plan.cg == 2 && plan.bn == 256) return launch_shape<2, 256, A_MN, B_MN>(p, plan, a, stream);
  if (plan.cg == 2) return launch_shape<2, 128, A_MN, B_MN>(p, plan, a, stream);
  return launch_shape<1, 128, A_MN, B_MN>(p, plan, a, stream);
}

void set_vec(Epilogue* e) {
  auto ok = [](const void* p, int64_t ld, uintptr_t bytes) {
    return p == nullptr || (aligned(p, bytes) && ld % 4 == 0);
  };
  e->vec = ok(e->bias, 0, 8) && ok(e->pre, e->ldp, 8) && ok(e->residual, e->ldr, 8) &&
           ok(e->slope_of, e->lds, 8) && ok(e->out, e->ldo, e->out_f32 ? 16 : 8);
}

cudaError_t launch_product(Product p, Space space, int withhold, cudaStream_t stream) {
  cudaError_t err = make_tileable(&p.a, &space, stream);
  if (err == cudaSuccess) err = make_tileable(&p.b, &space, stream);
  if (err != cudaSuccess) return err;
  set_vec(&p.e);
  const Plan plan = plan_product(p.rows, p.cols, p.depth);
  ProductArgs a{};
  a.e = p.e;
  a.rows = p.rows;
  a.cols = p.cols;
  a.splits = plan.splits;
  a.steps = static_cast<int32_t>((p.depth + kDepth - 1) / kDepth);
  a.withhold = withhold;
  JoinArgs join{};
  if (plan.splits > 1) {
    join.ld = round_up(p.cols, 4);
    join.stride = p.rows * join.ld;
    float* parts = static_cast<float*>(space.take(parts_bytes(plan, p.rows, p.cols)));
    join.parts = parts;
    join.splits = plan.splits;
    join.rows = p.rows;
    join.cols = p.cols;
    join.e = p.e;
    a.e = Epilogue{};
    a.e.out = parts;
    a.e.ldo = join.ld;
    a.e.out_f32 = 1;
    a.e.vec = 1;
    a.split_stride = join.stride;
  }
  err = p.a_mn   ? launch_majors<true, true>(p, plan, a, stream)
        : p.b_mn ? launch_majors<false, true>(p, plan, a, stream)
                 : launch_majors<false, false>(p, plan, a, stream);
  if (err != cudaSuccess || plan.splits == 1) return err;
  const int64_t blocks = (p.rows * (join.ld / 4) + 255) / 256;
  linear_join_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(join);
  return cudaGetLastError();
}

// Workspace of a product whose operands may both have to be laid out anew.
int64_t product_bytes(const Stored& a, const Stored& b, int64_t rows, int64_t cols, int64_t depth) {
  return copy_bytes(a) + copy_bytes(b) + parts_bytes(plan_product(rows, cols, depth), rows, cols);
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

__global__ void __launch_bounds__(256) linear_slope_kernel(const __grid_constant__ SlopeArgs a) {
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

}  // namespace

int read_and_clear_linear_status(int* status) {
  take_linear_status_kernel<<<1, 1, 0, 0>>>();
  if (cudaGetLastError() != cudaSuccess) return -1;
  int v = 0;  // the copy is ordered after the kernel on the legacy default stream
  if (cudaMemcpyFromSymbol(&v, g_linear_status_taken, sizeof(int)) != cudaSuccess) return -1;
  *status = v;
  return 0;
}

int64_t linear_workspace(const zero_linear_t& s, bool backward) {
  const Stored x{nullptr, s.rows, s.in, 0}, w{nullptr, s.out, s.in, 0}, z{nullptr, s.rows, s.out, 0}, none{nullptr, 0, 0, 0};
  if (!backward) return product_bytes(x, w, s.rows, s.out, s.in);
  // dz is laid out once and taken by both products, one after the other
  const int64_t dx = product_bytes(none, w, s.rows, s.in, s.out);
  const int64_t dw = product_bytes(none, x, s.out, s.in, s.rows);
  return copy_bytes(z) + (dx > dw ? dx : dw);
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
  return launch_product(p, {static_cast<char*>(L.workspace)}, L.withhold, L.stream);
}

cudaError_t launch_linear_backward(const LinearBackwardLaunch& L) {
  (void)cudaGetLastError();
  const zero_linear_t& s = L.s;
  Stored dz{L.dy, s.rows, s.out, s.ldy};
  Space space{static_cast<char*>(L.workspace)};
  if (L.act != ZERO_ACT_NONE || L.dbias != nullptr) {
    SlopeArgs a{L.dy, L.pre, s.ldy, s.ldp, s.rows, s.out, L.act, nullptr, 0, L.dbias,
                L.grad_f32, L.accumulate};
    if (L.act != ZERO_ACT_NONE && (L.dx != nullptr || L.dw != nullptr)) {
      a.dz = static_cast<uint16_t*>(space.take(copy_bytes(dz)));
      a.ldz = round_up(s.out, 8);
      dz.p = a.dz;
      dz.ld = a.ldz;
    }
    linear_slope_kernel<<<static_cast<unsigned>((s.out + 31) / 32), 256, 0, L.stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (s.rows == 0) {
    if (L.dw == nullptr || L.accumulate) return cudaSuccess;
    return cudaMemset2DAsync(L.dw, s.lddw * (L.grad_f32 ? 4 : 2), 0, s.in * (L.grad_f32 ? 4 : 2),
                             s.out, L.stream);
  }
  if (L.dx != nullptr || L.dw != nullptr) {
    const cudaError_t e = make_tileable(&dz, &space, L.stream);
    if (e != cudaSuccess) return e;
  }
  if (L.dx != nullptr) {
    Product p{};
    p.a = dz;
    p.b = {L.w, s.out, s.in, s.ldw};
    p.b_mn = true;
    p.rows = s.rows;
    p.cols = s.in;
    p.depth = s.out;
    p.e.slope_act = L.act_in;
    p.e.slope_of = L.act_in != ZERO_ACT_NONE ? L.pre_in : nullptr;
    p.e.lds = s.ldpi;
    p.e.out = L.dx;
    p.e.ldo = s.lddx;
    const cudaError_t e = launch_product(p, space, L.withhold, L.stream);
    if (e != cudaSuccess) return e;
  }
  if (L.dw != nullptr) {
    Product p{};
    p.a = dz;
    p.a_mn = true;
    p.b = {L.x, s.rows, s.in, s.ldx};
    p.b_mn = true;
    p.rows = s.out;
    p.cols = s.in;
    p.depth = s.rows;
    p.e.out = L.dw;
    p.e.ldo = s.lddw;
    p.e.out_f32 = L.grad_f32;
    p.e.accumulate = L.accumulate;
    return launch_product(p, space, L.withhold, L.stream);
  }
  return cudaSuccess;
}

}  // namespace zeroadam
