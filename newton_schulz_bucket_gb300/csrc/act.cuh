// Activations of the layer operators and their slopes, in fp32.
//
// kFast (16-bit tensors) takes the hardware exponential and division.  The
// exponential's relative error grows with its argument, about 1.2 units in the
// last place (2^-23) for each 1: 1e-5 at the largest argument that does not
// underflow, far below the 2^-9 (bf16) or 2^-12 (fp16) of the store.  fp32 tensors
// take the full-precision functions.
//
// GELU needs Phi(z) = (1 + erf(z / sqrt 2)) / 2 to a relative error, not an
// absolute one: that sum cancels for negative z (off by 4% at -5, zero below -5.6,
// where z Phi(z) is still a normal number of bf16 and fp32).  See normal_cdf.
#pragma once

#include <cuda_runtime.h>

#include "ops.h"

namespace muon {

template <bool kFast>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (kFast) return __fdividef(1.f, 1.f + __expf(-v));
  return 1.f / (1.f + expf(-v));
}

constexpr float kInvSqrt2Pi = 0.39894228040143267794f;      // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286535588f;     // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// Phi(z), and e = exp(-z^2 / 2), which the slope needs too.  With x = |z| and t = 1 /
// (1 + 0.2625 x), Phi(-x) = e t P(t): the quotient Phi(-x) / (e t) is smooth in t down
// to t = 0 (x = infinity).  P is its polynomial of least relative error on 0 <= x <=
// 14.5, where e underflows, found by reweighted least squares in 64 bits: degree 6 is
// within 8.4e-7 (16-bit tensors), degree 8 within 2.1e-8.  Rounding z^2 / 2 adds up to z^2
// 2^-25.  One exponential and one division: 4096 tokens, [4096, 16384], bf16 308 us and
// 684 back (the same box: erff 313 and 705, erfcf 351 and 756).
template <bool kFast>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float u = -0.5f * z * z, d = fmaf(0.2625f, fabsf(z), 1.f);
  e = kFast ? __expf(u) : expf(u);
  const float t = kFast ? __fdividef(1.f, d) : 1.f / d;
  float q;
  if constexpr (kFast) {
    q = -0.06988801807f;
    q = fmaf(q, t, 0.2101149708f);
    q = fmaf(q, t, -0.08346113563f);
    q = fmaf(q, t, 0.1524195522f);
    q = fmaf(q, t, 0.07887178659f);
    q = fmaf(q, t, 0.1073758826f);
    q = fmaf(q, t, 0.1045673862f);
  } else {
    q = 0.03052652441f;
    q = fmaf(q, t, -0.1477536857f);
    q = fmaf(q, t, 0.2325934619f);
    q = fmaf(q, t, -0.1309272498f);
    q = fmaf(q, t, 0.1474449188f);
    q = fmaf(q, t, 0.05656810477f);
    q = fmaf(q, t, 0.1026348621f);
    q = fmaf(q, t, 0.1041646823f);
    q = fmaf(q, t, 0.1047483608f);
  }
  const float tail = e * t * q;
  return z < 0.f ? tail : 1.f - tail;
}

// (1 + tanh u) / 2 = sigmoid(2 u), so GELU_TANH is z * sigmoid(2 u).
template <bool kFast>
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case ACT_SILU: return z * sigmoid<kFast>(z);
    case ACT_GELU: {
      float e;
      return z * normal_cdf<kFast>(z, e);
    }
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
      float e;
      const float cdf = normal_cdf<kFast>(z, e);
      return cdf + z * kInvSqrt2Pi * e;
    }
    case ACT_GELU_TANH: {
      const float p = sigmoid<kFast>(2.f * kSqrt2OverPi * (z + kTanhCubic * z * z * z));
      // z^2 comes in last, on what is zero where it would overflow (infinity times 0
      // would be NaN)
      const float a = z * (p * (1.f - p));
      return fmaf(2.f * kSqrt2OverPi, fmaf(3.f * kTanhCubic, z * (z * a), a), p);
    }
    default: return 1.f;
  }
}

}  // namespace muon
