// Activations of include/moe_experts.h's products and their derivatives, FP32.
#pragma once

#include "common.h"

namespace moe {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActSwiglu = 4 };

__device__ __forceinline__ float sigmoid_f32(float z) { return 1.0f / (1.0f + expf(-z)); }

// Phi(z), the normal distribution's: by erfc of the half that does not cancel.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f || z != z ? z : 0.0f;   // NaN stays
  else if constexpr (ACT == kActSilu) return z * sigmoid_f32(z);
  else if constexpr (ACT == kActGelu) return z * normal_cdf(z);
  else return z;
}

// d act / dz (relu'(0) = 0).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  else if constexpr (ACT == kActSilu) {
    const float e = sigmoid_f32(z);
    return e * fmaf(z, 1.0f - e, 1.0f);
  } else if constexpr (ACT == kActGelu) {
    return fmaf(z, 0.39894228040143268f * expf(-0.5f * z * z), normal_cdf(z));
  } else return 1.0f;
}

}  // namespace moe
