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

// 2^x and 1/x of the special-function unit: 2 ulp and 1 ulp; results below the
// least normal number are 0, 1/inf is 0.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations at a time.
struct Pair {
  uint64_t v;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ void split(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.v));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

// gelu's tanh form is z times the logistic function of 2u, u = sqrt(2/pi) (z + a z^3),
// since (1 + tanh u) / 2 = 1 / (1 + exp(-2u)); silu is z times that of z.  Both as
// p = 1 / (1 + 2^t), t = z (k0 + k1 z^2) with log2(e) and the sign in k0 and k1.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluA = 0.044715f;
constexpr float kGeluT0 = -kLog2e * kGelu2C, kGeluT1 = -kLog2e * kGelu2C * kGeluA;
// Where 2^t is inf or 0, p is 0 or 1 and z p (1 - p) is 0 for finite z.  An
// infinite z is kept from meeting 0 by these bounds, past which p is flat to the
// last bit of fp32; a NaN comes through p.
constexpr float kActMost = 3.402823466e38f, kActFlat = 104.0f;

template <int ACT>
__device__ __forceinline__ void logistic2(float z0, float z1, Pair& p) {
  const Pair z = pair(z0, z1);
  Pair t;
  if constexpr (ACT == ZERO_ACT_GELU)
    t = z * fma2(z * z, pair(kGeluT1, kGeluT1), pair(kGeluT0, kGeluT0));
  else
    t = z * pair(-kLog2e, -kLog2e);
  float t0, t1;
  split(t, t0, t1);
  split(pair(fast_exp2(t0), fast_exp2(t1)) + pair(1.0f, 1.0f), t0, t1);
  p = pair(fast_inverse(t0), fast_inverse(t1));
}

// act of two sums, in place.
template <int ACT>
__device__ __forceinline__ void act_value2(float& z0, float& z1) {
  if constexpr (ACT == ZERO_ACT_RELU) {
    z0 = z0 < 0.0f ? 0.0f : z0;
    z1 = z1 < 0.0f ? 0.0f : z1;
  } else if constexpr (ACT != ZERO_ACT_NONE) {
    Pair p;
    logistic2<ACT>(z0, z1, p);
    split(pair(fmaxf(z0, -kActMost), fmaxf(z1, -kActMost)) * p, z0, z1);
  }
}

// x0 and x1 times act' at z0 and z1:
//   silu' = p + z (p - p^2),  gelu' = p + z (p - p^2) 2 sqrt(2/pi) (1 + 3 a z^2)
template <int ACT>
__device__ __forceinline__ void times_slope2(float& x0, float& x1, float z0, float z1) {
  if constexpr (ACT == ZERO_ACT_RELU) {
    x0 *= z0 > 0.0f ? 1.0f : 0.0f;
    x1 *= z1 > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT != ZERO_ACT_NONE) {
    Pair p;
    logistic2<ACT>(z0, z1, p);
    Pair z = pair(fminf(fmaxf(z0, -kActFlat), kActFlat), fminf(fmaxf(z1, -kActFlat), kActFlat));
    if constexpr (ACT == ZERO_ACT_GELU)
      z = z * fma2(z * z, pair(3.0f * kGeluA * kGelu2C, 3.0f * kGeluA * kGelu2C),
                   pair(kGelu2C, kGelu2C));
    const Pair flat = fma2(p * pair(-1.0f, -1.0f), p, p);  // p - p^2
    split(pair(x0, x1) * fma2(z, flat, p), x0, x1);
  }
}

__device__ __forceinline__ float act_value(float z, int act) {
  float unused = 0.0f;
  if (act == ZERO_ACT_GELU) act_value2<ZERO_ACT_GELU>(z, unused);
  else if (act == ZERO_ACT_SILU) act_value2<ZERO_ACT_SILU>(z, unused);
  else if (act == ZERO_ACT_RELU) act_value2<ZERO_ACT_RELU>(z, unused);
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  float slope = 1.0f, unused = 0.0f;
  if (act == ZERO_ACT_GELU) times_slope2<ZERO_ACT_GELU>(slope, unused, z, 0.0f);
  else if (act == ZERO_ACT_SILU) times_slope2<ZERO_ACT_SILU>(slope, unused, z, 0.0f);
  else if (act == ZERO_ACT_RELU) times_slope2<ZERO_ACT_RELU>(slope, unused, z, 0.0f);
  return slope;
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
  const float* scale;        // gradients: multiplies the sum first, one number on the device
  const float* row_scale;    // and one for each row (bf16 alone); 0: the row is 0 whatever its sum is
  int32_t vec;               // every matrix's base and pitch are multiples of 16 bytes
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
    for (int c = 0; c < 8; c += 2) act_value2<ZERO_ACT_GELU>(x[c], x[c + 1]);
  } else if (act == ZERO_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < 8; c += 2) act_value2<ZERO_ACT_SILU>(x[c], x[c + 1]);
  } else if (act == ZERO_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < 8; c += 2) act_value2<ZERO_ACT_RELU>(x[c], x[c + 1]);
  }
}
__device__ __forceinline__ void times_slope8(float x[8], const uint4 at, int act) {
  float z[8];
  bf16x8(at, z);
  if (act == ZERO_ACT_GELU) {
#pragma unroll
    for (int c = 0; c < 8; c += 2) times_slope2<ZERO_ACT_GELU>(x[c], x[c + 1], z[c], z[c + 1]);
  } else if (act == ZERO_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < 8; c += 2) times_slope2<ZERO_ACT_SILU>(x[c], x[c + 1], z[c], z[c + 1]);
  } else if (act == ZERO_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < 8; c += 2) times_slope2<ZERO_ACT_RELU>(x[c], x[c + 1], z[c], z[c + 1]);
  }
}

}  // namespace zeroadam
