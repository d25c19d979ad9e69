// adamw_tensors.cu -- AdamW over a list of tensors, its 8-bit moments, and the
// global gradient norm, on sm_103a.
//
// All three stream every element once and do little with it, so they are bound
// by HBM bandwidth; what a list adds is that a block has to find its tensor.
// The tensors' descriptors travel in the kernel's arguments (constant memory:
// no table in device memory to lay out, nothing to free, captured by a graph as
// they are), and a launch covers as many tensors as fit there.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "train_ops.cuh"

namespace zeroadam {
namespace {

constexpr int kThreads = 256;
// Elements of a tile: each warp's, one moment block of 256 or several in a row,
// so that finding the tensor (10 to 50 instructions a warp) does not count.
constexpr int kBlocksOfWarp32 = 1, kBlocksOfWarp8 = 1, kBlocksOfWarpMoments = 2;
__host__ __device__ constexpr int tile_of_blocks(int blocks) { return kThreads * 8 * blocks; }

__device__ __forceinline__ float bf16_value(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// One step of O'Neill's 32-bit permuted congruential generator (RXS-M-XS),
// used as a hash (Jarzynski and Olano, "Hash Functions for GPU Rendering").
__host__ __device__ __forceinline__ uint32_t pcg_hash(uint32_t x) {
  x = x * 747796405u + 2891336453u;
  x = ((x >> ((x >> 28) + 4)) ^ x) * 277803737u;
  return (x >> 22) ^ x;
}

// Index of the tensor that holds `tile`: the last with tile0 <= tile, from `low`
// on.  The tensors' first tiles are an array of their own, which stays in the
// constant cache where the descriptors around them would not.
__device__ __forceinline__ int find_tensor(const int32_t* tile0, int count, int tile, int low) {
  int high = count;  // tile0[low] <= tile < tile0[high]
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if (tile0[mid] <= tile) low = mid; else high = mid;
  }
  return low;
}

// How a warp's 32 lanes take 256 elements, 8 each.
enum Access {
  kScalar,   // elements lane + 32 j, one by one; those outside the tensor are 0
  kVector,   // elements 8 lane + j, in 16-byte accesses
  // A moment block of a tensor whose buffers all begin `shift` elements past a
  // 16-byte boundary (tensors packed in flat vectors): elements 8 lane + j - shift,
  // so that vectors are aligned; the first lane's elements below 0 are instead the
  // block's last ones, 256 higher, and it takes its elements one by one.
  kRotated,
};

struct Span {
  int64_t base;  // first element
  int64_t n;     // of the tensor
  int lane, shift;
  // a lane's first element (kVector, kRotated)
  template <Access A>
  __device__ __forceinline__ int64_t at() const {
    return base + 8 * lane - (A == kRotated ? shift : 0);
  }
  // element j of the lane
  template <Access A>
  __device__ __forceinline__ int64_t element(int j) const {
    if (A == kScalar) return base + lane + 32 * j;
    const int64_t e = at<A>() + j;
    return A == kRotated && lane == 0 && j < shift ? e + 256 : e;
  }
  __device__ __forceinline__ bool inside(int64_t e) const {
    return static_cast<uint64_t>(e) < static_cast<uint64_t>(n);
  }
};

__device__ __forceinline__ void vector_f32(const float* p, float x[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void vector_bf16(const uint16_t* p, float x[8]) {
  const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

template <Access A>
__device__ __forceinline__ void load_f32(const float* p, const Span& s, float x[8]) {
  if (A == kVector || (A == kRotated && s.lane > 0)) {
    vector_f32(p + s.at<A>(), x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = s.element<A>(j);
      x[j] = A == kRotated || s.inside(e) ? __ldcs(p + e) : 0.0f;
    }
  }
}

template <Access A>
__device__ __forceinline__ void store_f32(float* p, const Span& s, const float x[8]) {
  if (A == kVector || (A == kRotated && s.lane > 0)) {
    float4* q = reinterpret_cast<float4*>(p + s.at<A>());
    __stcs(q, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(q + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = s.element<A>(j);
      if (A == kRotated || s.inside(e)) __stcs(p + e, x[j]);
    }
  }
}

template <Access A, bool GF32>
__device__ __forceinline__ void load_grad(const void* g, const Span& s, float x[8]) {
  if (GF32) {
    load_f32<A>(static_cast<const float*>(g), s, x);
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(g);
  if (A == kVector || (A == kRotated && s.lane > 0)) {
    vector_bf16(p + s.at<A>(), x);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = s.element<A>(j);
      x[j] = A == kRotated || s.inside(e) ? bf16_value(__ldcs(p + e)) : 0.0f;
    }
  }
}

template <Access A>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Span& s, const float x[8]) {
  if (A == kVector || (A == kRotated && s.lane > 0)) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bf16_bits(x[2 * j]) | (bf16_bits(x[2 * j + 1]) << 16);
    __stcs(reinterpret_cast<uint4*>(p + s.at<A>()), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = s.element<A>(j);
      if (A == kRotated || s.inside(e))
        __stcs(reinterpret_cast<unsigned short*>(p) + e,
               static_cast<unsigned short>(bf16_bits(x[j])));
    }
  }
}

// 8 codes as two words, code j in byte j % 4 of word j / 4.  (Codes have
// allocations of their own, so kRotated's are aligned without the shift: each
// lane takes its last bytes from the lane before it.)
template <Access A>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, const Span& s) {
  if (A == kScalar) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = s.element<A>(j);
      if (s.inside(e)) w[j / 4] |= static_cast<uint32_t>(__ldcs(p + e)) << (8 * (j % 4));
    }
    return make_uint2(w[0], w[1]);
  }
  uint2 r = __ldcs(reinterpret_cast<const uint2*>(p + s.base + 8 * s.lane));
  if (A == kRotated) {
    const uint64_t own = static_cast<uint64_t>(r.y) << 32 | r.x;
    const uint64_t before = __shfl_sync(0xffffffffu, own, (s.lane + 31) % 32);
    const uint64_t v = own << (8 * s.shift) | before >> (64 - 8 * s.shift);  // shift is 1 to 7
    r = make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
  }
  return r;
}

// The codes are the top bytes of c.
template <Access A>
__device__ __forceinline__ void store_codes(uint8_t* p, const Span& s, const uint32_t c[8]) {
  if (A == kScalar) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = s.element<A>(j);
      if (s.inside(e))
        __stcs(reinterpret_cast<unsigned char*>(p) + e, static_cast<unsigned char>(c[j] >> 24));
    }
    return;
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    w[k] = __byte_perm(__byte_perm(c[4 * k], c[4 * k + 1], 0x0073),
                       __byte_perm(c[4 * k + 2], c[4 * k + 3], 0x0073), 0x5410);
  if (A == kRotated) {
    const uint64_t own = static_cast<uint64_t>(w[1]) << 32 | w[0];
    const uint64_t after = __shfl_sync(0xffffffffu, own, (s.lane + 1) % 32);
    const uint64_t v = own >> (8 * s.shift) | after << (64 - 8 * s.shift);
    w[0] = static_cast<uint32_t>(v);
    w[1] = static_cast<uint32_t>(v >> 32);
  }
  __stcs(reinterpret_cast<uint2*>(p + s.base + 8 * s.lane), make_uint2(w[0], w[1]));
}

// ------------------------------------------------------------ 8-bit moments
//
// A code's bits, put 20 places up, are the bits of a binary32 number whose
// exponent field is the code's own: for m (4 exponent bits, top 15) that number
// is the value over 2^112 times the block's scale, for v (5 bits, top 31) over
// 2^96, and gradual underflow comes with binary32's own denormals.  So decoding
// is a shift and two exact products with powers of two, and encoding two such
// products, an integer addition of the random bits (whose carry is the rounding
// up) and a shift.
constexpr float kMUp = 0x1p112f, kMDown = 0x1p-112f;
constexpr float kVUp = 0x1p96f, kVDown = 0x1p-96f;

//
// The two products are one, with the same result, while their factors' product
// is a binary32 number itself: up to a scale of 2^15 (m) and 2^31 (v), which no
// moment of a working training step passes.  WIDE takes them one by one.
//
// What bounds the step is the integer pipe, of half the fp32 pipe's width, so
// shifts that can be are products, a code's place is reached by a byte
// permutation, the largest magnitude is taken three at a time, and a code's last
// cut is the permutation that packs it: 36 integer instructions an element were
// 5.9 TB/s on bf16 gradients.
//
// Code j of a word as the number over 2^112 (2^96) it stands for.
__device__ __forceinline__ float bits_of_v(uint32_t word, int j) {
  return __uint_as_float(__byte_perm(word, 0, 0x4044 | (j << 8)) * 16u);
}
__device__ __forceinline__ float bits_of_m(uint32_t word, int j) {
  const uint32_t t = __byte_perm(word, 0, 0x4044 | (j << 8)) * 16u;
  return __uint_as_float((t & 0x08000000u) * 15u + t);  // bit 27, the sign, to bit 31
}

__device__ __forceinline__ void decode8(uint2 mc, uint2 vc, float ms, float vs, float m[8],
                                        float v[8]) {
  const uint32_t mw[2] = {mc.x, mc.y}, vw[2] = {vc.x, vc.y};
  if (ms <= 0x1p15f && vs <= 0x1p31f) {
    const float mu = ms * kMUp, vu = vs * kVUp;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = __fmul_rn(bits_of_m(mw[j / 4], j % 4), mu);
      v[j] = __fmul_rn(bits_of_v(vw[j / 4], j % 4), vu);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = __fmul_rn(__fmul_rn(bits_of_m(mw[j / 4], j % 4), kMUp), ms);
      v[j] = __fmul_rn(__fmul_rn(bits_of_v(vw[j / 4], j % 4), kVUp), vs);
    }
  }
}

// The bits of the largest magnitude; a NaN's among them are larger than any.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t top_of(const float x[8]) {
  const float a = max_abs3(max_abs3(x[0], x[1], x[2]), x[3], x[4]);
  return __float_as_uint(max_abs3(max_abs3(a, x[5], x[6]), x[7], x[7])) & 0x7fffffffu;
}

// A block's scale from the bits of its largest magnitude: the exponent after
// rounding up to 4 significant bits, so that no code overflows by rounding up.
struct BlockScale {
  float scale, inverse;
  uint32_t field;  // exponent field of the scale
  bool fine;       // false: an infinity or NaN among the block's values
};
__device__ __forceinline__ BlockScale block_scale(uint32_t top) {
  uint32_t e = (top + 0xfffffu) >> 23;
  e = e < 1u ? 1u : e > 253u ? 253u : e;
  BlockScale b;
  b.field = e;
  b.fine = top < 0x7f800000u;
  b.scale = b.fine ? __uint_as_float(e << 23) : __uint_as_float(0x7fffffffu);
  b.inverse = __uint_as_float((254u - e) << 23);
  return b;
}

// Codes in the top bytes of mc and vc.  Except at the end of the scales' range
// (WIDE), no code is past the largest: the scale saw to it.
// The random bits are those of elements first + step j, the first `wrap` of them
// 256 further on.
template <bool WIDE>
__device__ __forceinline__ void encode8(const float m[8], const float v[8], const BlockScale& mb,
                                        const BlockScale& vb, uint32_t first, uint32_t step,
                                        int wrap, uint32_t mc[8], uint32_t vc[8]) {
  const float md = mb.inverse * kMDown, vd = vb.inverse * kVDown;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = pcg_hash(first + step * j + (j < wrap ? 256u : 0u));
    const float a = fabsf(m[j]), b = fabsf(v[j]);
    const float s = WIDE ? __fmul_rn(__fmul_rn(a, mb.inverse), kMDown) : __fmul_rn(a, md);
    const float t = WIDE ? __fmul_rn(__fmul_rn(b, vb.inverse), kVDown) : __fmul_rn(b, vd);
    uint32_t x = __float_as_uint(s) + ((u >> 12) & 0xffff0u) + 8u;
    uint32_t y = __float_as_uint(t) + ((u * 16u) & 0xffff0u) + 8u;
    if (WIDE) {
      x = x < 0x07ffffffu ? x : 0x07ffffffu;
      y = y < 0x0fffffffu ? y : 0x0fffffffu;
    }
    mc[j] = ((x * 16u) & 0x7fffffffu) | (__float_as_uint(m[j]) & 0x80000000u);
    vc[j] = y * 16u;
  }
  if (!mb.fine) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mc[j] = 0;
  }
  if (!vb.fine) {
#pragma unroll
    for (int j = 0; j < 8; ++j) vc[j] = 0;
  }
}

struct AdamwDesc {
  const void* grad;
  float* master;
  uint16_t* param;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t numel;
  float keep;    // 1 - lr * weight_decay
  uint32_t key;  // of the random bits
  int32_t access;  // Access, where a warp's elements are all in the tensor
  int32_t shift;   // elements from the 16-byte boundary before the tensor to its start
};

template <int CAP>
struct AdamwArgs {
  int32_t tile0[CAP];  // first tile of each tensor
  AdamwDesc t[CAP];
  AdamwScalars s;
  const float* grad_scale;
  int32_t count, tiles;
};

// One element; the sums and products that m and v are made of are rounded one
// by one, as the flat step's are, so that codes and moments have one value.
__device__ __forceinline__ void adamw_element(float g, const AdamwScalars& s, float keep, float& w,
                                              float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(s.omb1, g));
  v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(s.omb2, g), g));
  // the root and the inverse of the special-function unit, 1 to 2 ulp each: the
  // correctly rounded ones took a quarter of the 8-bit step's time.  (The inverse
  // takes denominators below the least normal number, which only eps = 0 and v = 0
  // give, as 0, and is 0 past 2^126.)
  float root, inverse;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inverse) : "f"(root * s.inv_root + s.eps));
  w = w * keep - s.size * m * inverse;
}

// 8 elements per thread; with 8-bit moments a warp's 256 are one moment block.
template <Access A, bool GF32, bool EIGHT>
__device__ __forceinline__ void adamw_tile(const AdamwDesc& t, const AdamwScalars& s, float clip,
                                           bool clipped, int64_t base, int lane) {
  const Span at{base, t.numel, lane, t.shift};
  float g[8], w[8], m[8], v[8];
  load_grad<A, GF32>(t.grad, at, g);
  load_f32<A>(t.master, at, w);
  if constexpr (EIGHT) {
    const int64_t block = base / ZERO_MOMENT_BLOCK;
    const uint2 mc = load_codes<A>(static_cast<const uint8_t*>(t.m), at);
    const uint2 vc = load_codes<A>(static_cast<const uint8_t*>(t.v), at);
    decode8(mc, vc, t.m_scale[block], t.v_scale[block], m, v);
  } else {
    load_f32<A>(static_cast<const float*>(t.m), at, m);
    load_f32<A>(static_cast<const float*>(t.v), at, v);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (clipped) g[j] = __fmul_rn(g[j], clip);
    adamw_element(g[j], s, t.keep, w[j], m[j], v[j]);
  }
  store_f32<A>(t.master, at, w);
  if (t.param != nullptr) store_bf16<A>(t.param, at, w);
  if constexpr (EIGHT) {
    const int64_t block = base / ZERO_MOMENT_BLOCK;
    if (A == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!at.inside(at.element<A>(j))) m[j] = v[j] = 0.0f;  // no element: no part in the scale
    }
    const uint32_t mtop = __reduce_max_sync(0xffffffffu, top_of(m));
    const uint32_t vtop = __reduce_max_sync(0xffffffffu, top_of(v));
    const BlockScale mb = block_scale(mtop), vb = block_scale(vtop);
    const uint32_t key = t.key + static_cast<uint32_t>(base >> 32) * 0x9E3779B9u;
    const int64_t e = A == kScalar ? base + lane : at.at<A>();
    const uint32_t first = static_cast<uint32_t>(e) + key;
    constexpr uint32_t step = A == kScalar ? 32 : 1;
    const int wrap = A == kRotated && lane == 0 ? t.shift : 0;
    uint32_t mc[8], vc[8];
    if (mb.field <= 127 + 14 && vb.field <= 127 + 30)
      encode8<false>(m, v, mb, vb, first, step, wrap, mc, vc);
    else
      encode8<true>(m, v, mb, vb, first, step, wrap, mc, vc);
    store_codes<A>(static_cast<uint8_t*>(t.m), at, mc);
    store_codes<A>(static_cast<uint8_t*>(t.v), at, vc);
    if (lane == 0) {
      t.m_scale[block] = mb.scale;
      t.v_scale[block] = vb.scale;
    }
  } else {
    store_f32<A>(static_cast<float*>(t.m), at, m);
    store_f32<A>(static_cast<float*>(t.v), at, v);
  }
}

// fp32 moments: a block a tile, in the order of memory (a persistent grid, whose
// blocks drift apart, streamed 5.9 TB/s where this does 7.1, 8e8 elements).
// 8-bit moments: a block's beginning counts, so at most 64 blocks an SM take
// tiles in turn (1, 4 or 16 tiles in a row to a block: 5 to 20 % slower).
// Tensors packed in flat vectors at any element (matrices of 12 layers, 1021
// wide): fp32 moments 7.1 TB/s as well (element by element: 5.1), 8-bit moments
// in the rotated order 4.2 (element by element: 3.6; with the first lane's
// elements handed on by shuffles instead of taken one by one: 4.0).
constexpr int kBlocksPerSm = 64;

template <int CAP, bool GF32, bool EIGHT>
__global__ void __launch_bounds__(kThreads, EIGHT ? 6 : 3)
    adamw_tensors_kernel(const __grid_constant__ AdamwArgs<CAP> a) {
  const bool clipped = a.grad_scale != nullptr;
  const float clip = clipped ? *a.grad_scale : 1.0f;
  constexpr int kBlocks = EIGHT ? kBlocksOfWarp8 : kBlocksOfWarp32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int ti = 0;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    ti = find_tensor(a.tile0, a.count, tile, ti);
    const AdamwDesc& t = a.t[ti];
    int64_t base = static_cast<int64_t>(tile - a.tile0[ti]) * tile_of_blocks(kBlocks) + 256 * warp;
    if constexpr (EIGHT) {
#pragma unroll 1
      for (int k = 0; k < kBlocks; ++k, base += tile_of_blocks(1)) {
        if (base >= t.numel) break;  // the same for the whole warp
        if (t.access == kVector && base + 256 <= t.numel)
          adamw_tile<kVector, GF32, true>(t, a.s, clip, clipped, base, lane);
        else if (t.access == kRotated && base + 256 <= t.numel)
          adamw_tile<kRotated, GF32, true>(t, a.s, clip, clipped, base, lane);
        else
          adamw_tile<kScalar, GF32, true>(t, a.s, clip, clipped, base, lane);
      }
    } else {
      base -= t.shift;  // tiles are counted from the 16-byte boundary before the tensor
      if (base >= t.numel) continue;
      if (t.access == kVector && base >= 0 && base + 256 <= t.numel)
        adamw_tile<kVector, GF32, false>(t, a.s, clip, clipped, base, lane);
      else
        adamw_tile<kScalar, GF32, false>(t, a.s, clip, clipped, base, lane);
    }
  }
}

struct MomentsDesc {
  const uint8_t* codes;
  const float* scale;
  float* out;
  int64_t numel;
  int32_t is_m, vec;
};

template <int CAP>
struct MomentsArgs {
  int32_t tile0[CAP];
  MomentsDesc t[CAP];
  int32_t count, tiles;
};

template <Access A>
__device__ __forceinline__ void moments_tile(const MomentsDesc& t, int64_t base, int lane) {
  const float scale = t.scale[base / ZERO_MOMENT_BLOCK];
  const Span at{base, t.numel, lane, 0};
  const uint2 c = load_codes<A>(t.codes, at);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? c.x : c.y;
    x[j] = __fmul_rn(t.is_m ? __fmul_rn(bits_of_m(w, j % 4), kMUp) : __fmul_rn(bits_of_v(w, j % 4), kVUp),
                     scale);
  }
  if (A == kVector)  // a lane's 32 bytes at once: two halves took 1,331 us where this takes 1,211 (8e8)
    asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(x[0]), "f"(x[1]),
                 "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]),
                 "l"(t.out + at.at<A>())
                 : "memory");
  else
    store_f32<A>(t.out, at, x);
}

// A block a tile, in the order of memory.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    adamw_moments_kernel(const __grid_constant__ MomentsArgs<CAP> a) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, tile = blockIdx.x;
  const int ti = find_tensor(a.tile0, a.count, tile, 0);
  const MomentsDesc& t = a.t[ti];
  int64_t base = static_cast<int64_t>(tile - a.tile0[ti]) * tile_of_blocks(kBlocksOfWarpMoments) +
                 256 * warp;
#pragma unroll 1
  for (int k = 0; k < kBlocksOfWarpMoments; ++k, base += tile_of_blocks(1)) {
    if (base >= t.numel) return;
    if (t.vec && base + 256 <= t.numel) moments_tile<kVector>(t, base, lane);
    else moments_tile<kScalar>(t, base, lane);
  }
}

// ------------------------------------------------------------------- norm

struct NormDesc {
  const void* grad;
  int64_t numel;
  int64_t shift;  // elements between the 16-byte boundary before the tensor and its start
};

constexpr int kNormTile = kThreads * 64;  // elements

template <int CAP>
struct NormArgs {
  int32_t tile0[CAP];
  NormDesc t[CAP];
  int32_t count, tiles;
  int32_t slot0, slots;  // this launch's first place in the workspace; places of all launches
  float max_norm;
  float* out;
  uint32_t* ticket;
  double* partial;
};

// The sum of a thread's up to 64 squares in fp32, its tiles and all else in
// fp64.  Vectors are counted from the 16-byte boundary at or before the
// tensor's start, so each is aligned whatever the tensor's address; the
// elements of the first and the last that are not the tensor's are left out.
template <int CAP, bool GF32>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ NormArgs<CAP> a) {
  constexpr int V = GF32 ? 4 : 8;  // elements of a 16-byte vector
  double sum = 0.0;
  int ti = 0;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    ti = find_tensor(a.tile0, a.count, tile, ti);
    const NormDesc& t = a.t[ti];
    const int64_t first = static_cast<int64_t>(tile - a.tile0[ti]) * kNormTile;
    const int64_t end = t.numel + t.shift;
    const char* p = static_cast<const char*>(t.grad) - t.shift * (GF32 ? 4 : 2);
    float acc = 0.0f;
    if (first >= t.shift && first + kNormTile <= end) {
      const uint4* q = reinterpret_cast<const uint4*>(p) + first / V;
#pragma unroll
      for (int r = 0; r < 64 / V; r += 8) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __ldcs(q + (r + j) * kThreads + threadIdx.x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (GF32) {
              const float f = __uint_as_float(w[k]);
              acc = fmaf(f, f, acc);
            } else {
              const float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
              acc = fmaf(lo, lo, acc);
              acc = fmaf(hi, hi, acc);
            }
          }
        }
      }
    } else {
      int64_t e = first + threadIdx.x;
      const int64_t stop = end < first + kNormTile ? end : first + kNormTile;
      for (; e < stop; e += kThreads) {
        if (e < t.shift) continue;
        const float f = GF32 ? __ldcs(reinterpret_cast<const float*>(p) + e)
                             : bf16_value(__ldcs(reinterpret_cast<const uint16_t*>(p) + e));
        acc = fmaf(f, f, acc);
      }
    }
    sum += static_cast<double>(acc);
  }

  __shared__ double part[kThreads / 32];
  __shared__ bool last;
  auto block_sum = [&](double x) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_down_sync(0xffffffffu, x, d);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0.0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) x += part[k];
    return x;
  };
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    a.partial[a.slot0 + blockIdx.x] = sum;
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == static_cast<uint32_t>(a.slots - 1);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  sum = 0.0;
  for (int k = threadIdx.x; k < a.slots; k += kThreads) sum += __ldcg(a.partial + k);
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(sqrt(sum));
    const float c = a.max_norm / (norm + 1e-6f);
    a.out[0] = norm;
    a.out[1] = c > 1.0f ? 1.0f : c;  // a NaN stays one
    *a.ticket = 0;
  }
}

int grid_of(int64_t tiles, int per_sm) {
  int sms = 0;
  if (device_sm_count(&sms) != 0) return 0;
  const int64_t most = static_cast<int64_t>(sms) * per_sm;
  return static_cast<int>(tiles < most ? tiles : most);
}

template <typename T>
bool aligned(const T* p, uintptr_t k) {
  return (reinterpret_cast<uintptr_t>(p) & (k - 1)) == 0;
}

// Kernel arguments hold at most 32,764 bytes.
constexpr int kAdamwMost = 384;

template <int CAP>
cudaError_t launch_adamw_chunk(const AdamwLaunch& L, const int32_t* index, int count) {
  AdamwArgs<CAP> a;
  static_assert(sizeof(a) <= 32764, "kernel arguments");
  int64_t tiles = 0;
  const uint32_t seed = pcg_hash(L.seed);
  for (int k = 0; k < count; ++k) {
    const zero_adamw_tensor_t& x = L.tensors[index[k]];
    AdamwDesc& t = a.t[k];
    t.grad = x.grad;
    t.master = x.master;
    t.param = static_cast<uint16_t*>(x.param_bf16);
    t.m = x.m;
    t.v = x.v;
    t.m_scale = x.m_scale;
    t.v_scale = x.v_scale;
    t.numel = x.numel;
    t.keep = static_cast<float>(1.0 - L.lr * x.weight_decay);
    t.key = pcg_hash(seed + static_cast<uint32_t>(index[k]));
    a.tile0[k] = static_cast<int32_t>(tiles);
    t.access = kScalar;
    t.shift = 0;
    for (int shift = 0; shift < 8 && t.access == kScalar; ++shift) {
      const auto fits = [&](const void* p, int size) {  // element -shift on a 16-byte boundary
        return p == nullptr || ((reinterpret_cast<uintptr_t>(p) - shift * size) & 15u) == 0;
      };
      if (!fits(t.grad, L.grad_f32 ? 4 : 2) || !fits(t.master, 4) || !fits(t.param, 2)) continue;
      if (L.eight ? !(aligned(t.m, 8) && aligned(t.v, 8)) : !(fits(t.m, 4) && fits(t.v, 4)))
        continue;
      t.access = L.eight && shift > 0 ? kRotated : kVector;
      t.shift = shift;
    }
    const int64_t per = tile_of_blocks(L.eight ? kBlocksOfWarp8 : kBlocksOfWarp32);
    tiles += (x.numel + (L.eight ? 0 : t.shift) + per - 1) / per;
  }
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  a.s = L.s;
  a.grad_scale = L.grad_scale;
  a.count = count;
  a.tiles = static_cast<int32_t>(tiles);
  const int grid = L.eight ? grid_of(tiles, kBlocksPerSm) : a.tiles;
  if (grid == 0) return cudaErrorNoDevice;
  if (L.grad_f32) {
    if (L.eight)
      adamw_tensors_kernel<CAP, true, true><<<grid, kThreads, 0, L.stream>>>(a);
    else
      adamw_tensors_kernel<CAP, true, false><<<grid, kThreads, 0, L.stream>>>(a);
  } else {
    if (L.eight)
      adamw_tensors_kernel<CAP, false, true><<<grid, kThreads, 0, L.stream>>>(a);
    else
      adamw_tensors_kernel<CAP, false, false><<<grid, kThreads, 0, L.stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamwLaunch& L) {
  (void)cudaGetLastError();
  int32_t index[kAdamwMost];
  for (int32_t i = 0; i < L.ntensors;) {
    int count = 0;
    for (; i < L.ntensors && count < kAdamwMost; ++i)
      if (L.tensors[i].numel > 0) index[count++] = i;
    if (count == 0) break;
    const cudaError_t e = count <= 16    ? launch_adamw_chunk<16>(L, index, count)
                          : count <= 160 ? launch_adamw_chunk<160>(L, index, count)
                                         : launch_adamw_chunk<kAdamwMost>(L, index, count);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_adamw_moments(const MomentsLaunch& L) {
  constexpr int kCap = 512;
  (void)cudaGetLastError();
  MomentsArgs<kCap> a;
  static_assert(sizeof(a) <= 32764, "kernel arguments");
  a.count = 0;
  int64_t tiles = 0;
  auto flush = [&]() -> cudaError_t {
    if (a.count == 0) return cudaSuccess;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = static_cast<int32_t>(tiles);
    adamw_moments_kernel<kCap><<<a.tiles, kThreads, 0, L.stream>>>(a);
    a.count = 0;
    tiles = 0;
    return cudaGetLastError();
  };
  for (int32_t i = 0; i < L.ntensors; ++i) {
    const zero_adamw_tensor_t& x = L.tensors[i];
    if (x.numel == 0) continue;
    for (int which = 0; which < 2; ++which) {
      float* const* out = which == 0 ? L.m_out : L.v_out;
      if (out == nullptr) continue;
      a.tile0[a.count] = static_cast<int32_t>(tiles);
      MomentsDesc& t = a.t[a.count++];
      t.codes = static_cast<const uint8_t*>(which == 0 ? x.m : x.v);
      t.scale = which == 0 ? x.m_scale : x.v_scale;
      t.out = out[i];
      t.numel = x.numel;
      t.is_m = which == 0;
      t.vec = aligned(t.codes, 8) && aligned(t.out, 32);
      constexpr int kPer = tile_of_blocks(kBlocksOfWarpMoments);
      tiles += (x.numel + kPer - 1) / kPer;
      if (a.count == kCap || tiles > INT32_MAX / 2) {
        const cudaError_t e = flush();
        if (e != cudaSuccess) return e;
      }
    }
  }
  return flush();
}

namespace {

template <int CAP>
cudaError_t launch_norm_chunk(const NormLaunch& L, const int32_t* index, int count, int slot0,
                              int slots, int grid) {
  NormArgs<CAP> a;
  static_assert(sizeof(a) <= 32764, "kernel arguments");
  int64_t tiles = 0;
  for (int k = 0; k < count; ++k) {
    NormDesc& t = a.t[k];
    t.grad = L.grads[index[k]];
    t.numel = L.numels[index[k]];
    a.tile0[k] = static_cast<int32_t>(tiles);
    t.shift = static_cast<int64_t>((reinterpret_cast<uintptr_t>(t.grad) & 15u) /
                                   (L.grad_f32 ? 4u : 2u));
    tiles += (t.numel + t.shift + kNormTile - 1) / kNormTile;
  }
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  a.count = count;
  a.tiles = static_cast<int32_t>(tiles);
  a.slot0 = slot0;
  a.slots = slots;
  a.max_norm = L.max_norm;
  a.out = L.out;
  a.ticket = static_cast<uint32_t*>(L.workspace);
  a.partial = reinterpret_cast<double*>(static_cast<char*>(L.workspace) + 16);
  if (L.grad_f32)
    grad_norm_kernel<CAP, true><<<grid, kThreads, 0, L.stream>>>(a);
  else
    grad_norm_kernel<CAP, false><<<grid, kThreads, 0, L.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grad_norm(const NormLaunch& L) {
  constexpr int kMost = 1024;
  (void)cudaGetLastError();
  // The blocks of each launch are settled first: the last block of all, whichever
  // launch it is in, adds up every block's part.
  int32_t left = 0;
  for (int32_t i = 0; i < L.ntensors; ++i) left += L.numels[i] > 0;
  const int launches = left == 0 ? 1 : (left + kMost - 1) / kMost;
  int grids[(ZERO_MAX_LIST + kMost - 1) / kMost];
  int64_t tiles = 0;
  int slots = 0;
  int launch = 0, count = 0;
  auto close = [&]() {
    int g = grid_of(tiles < 1 ? 1 : tiles, 4);
    if (g > kNormSlots / launches) g = static_cast<int>(kNormSlots / launches);
    grids[launch++] = g;
    slots += g;
    tiles = 0;
    count = 0;
  };
  for (int32_t i = 0; i < L.ntensors; ++i) {
    if (L.numels[i] == 0) continue;
    const int64_t shift = static_cast<int64_t>((reinterpret_cast<uintptr_t>(L.grads[i]) & 15u) /
                                               (L.grad_f32 ? 4u : 2u));
    tiles += (L.numels[i] + shift + kNormTile - 1) / kNormTile;
    if (++count == kMost) close();
  }
  if (count > 0 || launch == 0) close();
  if (grids[0] == 0) return cudaErrorNoDevice;
  int32_t index[kMost];
  int32_t i = 0;
  int slot0 = 0;
  for (int k = 0; k < launch; ++k) {
    count = 0;
    for (; i < L.ntensors && count < kMost; ++i)
      if (L.numels[i] > 0) index[count++] = i;
    const cudaError_t e =
        count <= 16    ? launch_norm_chunk<16>(L, index, count, slot0, slots, grids[k])
        : count <= 160 ? launch_norm_chunk<160>(L, index, count, slot0, slots, grids[k])
                       : launch_norm_chunk<kMost>(L, index, count, slot0, slots, grids[k]);
    if (e != cudaSuccess) return e;
    slot0 += grids[k];
  }
  return cudaSuccess;
}

}  // namespace zeroadam
