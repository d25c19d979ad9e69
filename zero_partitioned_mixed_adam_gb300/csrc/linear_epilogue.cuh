// linear_epilogue.cuh -- the activations, and what becomes of an fp32 sum of a
// linear map's product before it is stored.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "zeroadam.h"

namespace zeroadam {

__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// 1 / (1 + exp(-x)); exp(-x) = inf gives 0.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

// gelu's tanh form is z times the logistic function of 2u, u = sqrt(2/pi) (z + a z^3),
// since (1 + tanh u) / 2 = 1 / (1 + exp(-2u)).
//
// Past kActFlat the logistic function is 0 or 1 to the last bit of fp32, so the
// value is 0 or z and the slope 0 or 1; taking them as such also keeps infinite
// and huge z from meeting 0 * inf.  A NaN fails both comparisons and stays one.
constexpr float kActFlat = 104.0f;

__device__ __forceinline__ float act_value(float z, int act) {
  if (act == ZERO_ACT_NONE) return z;
  if (act == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if (fabsf(z) > kActFlat) return z > 0.0f ? z : 0.0f;
  return z * logistic(act == ZERO_ACT_GELU ? kGelu2C * (z + kGeluA * z * z * z) : z);
}

__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == ZERO_ACT_NONE) return 1.0f;
  if (act == ZERO_ACT_RELU || fabsf(z) > kActFlat) return z > 0.0f ? 1.0f : 0.0f;
  if (act == ZERO_ACT_GELU) {
    const float p = logistic(kGelu2C * (z + kGeluA * z * z * z));
    return p + z * p * (1.0f - p) * (kGelu2C * (1.0f + 3.0f * kGeluA * z * z));
  }
  const float p = logistic(z);
  return p * (1.0f + z * (1.0f - p));
}

// The epilogue of a product D[rows, cols]: what is added to, made of and
// multiplied with a sum before it is stored.  Pointers that are NULL leave
// their step out.
struct Epilogue {
  const uint16_t* bias;      // [cols]
  int32_t act;               // of the sum plus bias
  uint16_t* pre;             // the sum plus bias, stored
  int64_t ldp;
  const uint16_t* residual;  // added after the activation
  int64_t ldr;
  int32_t slope_act;         // multiplies by act'(slope_of)
  const uint16_t* slope_of;
  int64_t lds;
  void* out;                 // bf16, or fp32
  int64_t ldo;
  int32_t out_f32, accumulate;
  int32_t vec;               // 16-byte accesses: every matrix's base and pitch allow them
};

// ---- one element, any layout

__device__ __forceinline__ void epilogue_element(const Epilogue& e, int64_t i, int64_t j, float x) {
  if (e.bias != nullptr) x += bf16_at(e.bias + j);
  if (e.pre != nullptr) e.pre[i * e.ldp + j] = to_bf16(x);
  x = act_value(x, e.act);
  if (e.residual != nullptr) x += bf16_at(e.residual + i * e.ldr + j);
  if (e.slope_of != nullptr) x *= act_slope(bf16_at(e.slope_of + i * e.lds + j), e.slope_act);
  if (e.out_f32) {
    float* o = static_cast<float*>(e.out) + i * e.ldo + j;
    *o = e.accumulate ? *o + x : x;
  } else {
    uint16_t* o = static_cast<uint16_t*>(e.out) + i * e.ldo + j;
    *o = to_bf16(e.accumulate ? bf16_at(o) + x : x);
  }
}

// ---- 8 columns as one 16-byte vector of bf16

__device__ __forceinline__ void bf16x8(const uint4 r, float x[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[2 * c] = __uint_as_float(w[c] << 16);
    x[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 to_bf16x8(const float x[8]) {
  return make_uint4(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]), bf16x2_bits(x[4], x[5]),
                    bf16x2_bits(x[6], x[7]));
}
// One branch for the 8 of them.
__device__ __forceinline__ void act_value8(float x[8], int act) {
  if (act == ZERO_ACT_GELU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = act_value(x[c], ZERO_ACT_GELU);
  } else if (act == ZERO_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = act_value(x[c], ZERO_ACT_SILU);
  } else if (act == ZERO_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = act_value(x[c], ZERO_ACT_RELU);
  }
}
__device__ __forceinline__ void times_slope8(float x[8], const uint4 at, int act) {
  float z[8];
  bf16x8(at, z);
  if (act == ZERO_ACT_GELU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] *= act_slope(z[c], ZERO_ACT_GELU);
  } else if (act == ZERO_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] *= act_slope(z[c], ZERO_ACT_SILU);
  } else if (act == ZERO_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] *= act_slope(z[c], ZERO_ACT_RELU);
  }
}

}  // namespace zeroadam
