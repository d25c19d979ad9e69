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
  int32_t vec;               // 4 columns at a time: every matrix's base and pitch allow it
};

__device__ __forceinline__ float4 bf16x4(const uint2 r) {
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ uint2 to_bf16x4(const float x[4]) {
  return make_uint2(to_bf16(x[0]) | (static_cast<uint32_t>(to_bf16(x[1])) << 16),
                    to_bf16(x[2]) | (static_cast<uint32_t>(to_bf16(x[3])) << 16));
}

// What the epilogue reads of 4 columns (j a multiple of 4) of row i.
struct EpilogueInputs {
  float bias[4], residual[4], slope_of[4], old[4];
};

// n: how many of the 4 columns exist.
__device__ __forceinline__ void epilogue_load4(const Epilogue& e, int64_t i, int64_t j, int n,
                                               EpilogueInputs& in) {
  auto take = [&](const uint16_t* p, float x[4]) {
    if (e.vec && n == 4) {
      const float4 v = bf16x4(*reinterpret_cast<const uint2*>(p));
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = c < n ? bf16_at(p + c) : 0.0f;
    }
  };
  if (e.bias != nullptr) take(e.bias + j, in.bias);
  if (e.residual != nullptr) take(e.residual + i * e.ldr + j, in.residual);
  if (e.slope_of != nullptr) take(e.slope_of + i * e.lds + j, in.slope_of);
  if (e.accumulate) {
    if (!e.out_f32) {
      take(static_cast<const uint16_t*>(e.out) + i * e.ldo + j, in.old);
    } else {
      const float* p = static_cast<const float*>(e.out) + i * e.ldo + j;
      if (e.vec && n == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        in.old[0] = v.x; in.old[1] = v.y; in.old[2] = v.z; in.old[3] = v.w;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) in.old[c] = c < n ? p[c] : 0.0f;
      }
    }
  }
}

__device__ __forceinline__ void epilogue_store4(const Epilogue& e, int64_t i, int64_t j, int n,
                                                const EpilogueInputs& in, float x[4]) {
  auto put = [&](uint16_t* p) {
    if (e.vec && n == 4) {
      *reinterpret_cast<uint2*>(p) = to_bf16x4(x);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) p[c] = to_bf16(x[c]);
    }
  };
  if (e.bias != nullptr) {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] += in.bias[c];
  }
  if (e.pre != nullptr) put(e.pre + i * e.ldp + j);
  if (e.act != ZERO_ACT_NONE) {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = act_value(x[c], e.act);
  }
  if (e.residual != nullptr) {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] += in.residual[c];
  }
  if (e.slope_of != nullptr) {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] *= act_slope(in.slope_of[c], e.slope_act);
  }
  if (e.accumulate) {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] += in.old[c];
  }
  if (!e.out_f32) {
    put(static_cast<uint16_t*>(e.out) + i * e.ldo + j);
  } else {
    float* p = static_cast<float*>(e.out) + i * e.ldo + j;
    if (e.vec && n == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) p[c] = x[c];
    }
  }
}

}  // namespace zeroadam
