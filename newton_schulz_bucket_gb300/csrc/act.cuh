// Activations of the layer operators and their slopes, in fp32.
//
// kFast (16-bit tensors) takes the hardware exponential and division, whose
// relative error of about 1e-6 is far below the 2^-9 (bf16) or 2^-12 (fp16)
// of the store; fp32 tensors take the full-precision functions.
#pragma once

#include <cuda_runtime.h>

#include "ops.h"

namespace muon {

template <bool kFast>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (kFast) return __fdividef(1.f, 1.f + __expf(-v));
  return 1.f / (1.f + expf(-v));
}

constexpr float kSqrtHalf = 0.70710678118654752440f;        // 1 / sqrt 2
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;      // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286535588f;     // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// (1 + tanh u) / 2 = sigmoid(2 u), so GELU_TANH is z * sigmoid(2 u).
template <bool kFast>
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case ACT_SILU: return z * sigmoid<kFast>(z);
    case ACT_GELU: return 0.5f * z * (1.f + erff(z * kSqrtHalf));
    case ACT_GELU_TANH: return z * sigmoid<kFast>(2.f * kSqrt2OverPi * (z + kTanhCubic * z * z * z));
    default: return z;
  }
}

template <bool kFast>
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case ACT_SILU: {
      const float p = sigmoid<kFast>(z);
      return p * (1.f + z * (1.f - p));
    }
    case ACT_GELU: {
      const float g = kFast ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
      return 0.5f * (1.f + erff(z * kSqrtHalf)) + z * kInvSqrt2Pi * g;
    }
    case ACT_GELU_TANH: {
      const float p = sigmoid<kFast>(2.f * kSqrt2OverPi * (z + kTanhCubic * z * z * z));
      return p + 2.f * z * p * (1.f - p) * kSqrt2OverPi * (1.f + 3.f * kTanhCubic * z * z);
    }
    default: return 1.f;
  }
}

}  // namespace muon
