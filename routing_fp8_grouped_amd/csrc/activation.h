// Activations of include/moe_experts.h's products and their derivatives, FP32.
#pragma once

#include "common.h"

namespace moe {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActSwiglu = 4 };

// e^z by the hardware's 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float exp_f32(float z) { return __builtin_amdgcn_exp2f(1.44269504088896341f * z); }

// By the hardware's 2^x and reciprocal (an ulp each): within (4 + |z|) 2^-23 of
// the exact value, where what it goes into is rounded to 16 bits; 0 where it is
// below 2^-126, from z = -87.3 on, where z times it is at most 2^-119.
__device__ __forceinline__ float sigmoid_f32(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-z)); }

// Phi(z), the normal distribution's: for t = |z|, Phi(-t) = e^(-t^2/2) g(t) with
// g(t) = e^(t^2/2) erfc(t / sqrt 2) / 2 smooth and falling, so a polynomial of
// degree 8 in u = 1 / (1 + 0.23 t) is within 5.8e-8 of it (relative, t <= 14; a
// minimax fit made for this file; beyond, e^(-t^2/2) is 0).  No cancellation on
// the side that vanishes; in FP32 the exponent's rounding leaves 1.3e-6 of Phi
// for |z| < 6 and 4e-6 at 12.  15 operations where the library's erfc takes some
// 150, which made a gelu the longest part of a narrow product's epilogue.
__device__ __forceinline__ float normal_cdf(float z) {
  const float t = fabsf(z), u = __builtin_amdgcn_rcpf(fmaf(0.23f, t, 1.0f));
  float p = -7.84674808e-2f;
  p = fmaf(p, u, 2.90414214e-1f);
  p = fmaf(p, u, -2.78127104e-1f);
  p = fmaf(p, u, 3.01472902e-1f);
  p = fmaf(p, u, -3.29202376e-2f);
  p = fmaf(p, u, 1.19514063e-1f);
  p = fmaf(p, u, 8.5762918e-2f);
  p = fmaf(p, u, 9.23784599e-2f);
  p = fmaf(p, u, -2.7762424e-5f);
  const float q = p * exp_f32(-0.5f * t * t);
  return z < 0.0f ? q : 1.0f - q;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f || z != z ? z : 0.0f;   // NaN stays
  else if constexpr (ACT == kActSilu) return z * sigmoid_f32(z);
  else if constexpr (ACT == kActGelu) return z * normal_cdf(z);
  else return z;
}

// silu(g) u
__device__ __forceinline__ float glu_value(float g, float u) { return g * sigmoid_f32(g) * u; }

// d act / dz (relu'(0) = 0).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  else if constexpr (ACT == kActSilu) {
    const float e = sigmoid_f32(z);
    return e * fmaf(z, 1.0f - e, 1.0f);
  } else if constexpr (ACT == kActGelu) {
    return fmaf(z, 0.39894228040143268f * exp_f32(-0.5f * z * z), normal_cdf(z));
  } else return 1.0f;
}

}  // namespace moe
