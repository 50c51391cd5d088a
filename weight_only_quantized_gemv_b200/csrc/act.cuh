// Activation functions of the fused linear layers and their derivatives, on fp32 values.
//
//   relu       max(z, 0)                        derivative: 1 for z > 0, else 0
//   gelu       z Phi(z), Phi the normal CDF     Phi(z) + z phi(z)
//   gelu_tanh  z sigma(2 v), v = sqrt(2 / pi) (z + 0.044715 z^3)  (= z (1 + tanh v) / 2, in the
//              form that does not cancel for small or very negative v)
//   silu       z sigma(z)                       sigma(z) (1 + z (1 - sigma(z)))
#pragma once
#include "qlinear.h"

namespace qact {

__host__ __device__ constexpr bool act_ok(int act) { return act >= QL_ACT_NONE && act <= QL_ACT_SILU; }

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + e^-x), fast exponential and reciprocal (a few fp32 ulps): 0 and 1 at the far ends.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// Phi(z) and e^(-z^2 / 2), without branches: Abramowitz and Stegun 7.1.26,
// erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2), t = 1 / (1 + p x), x = |z| / sqrt 2, which is off by at
// most 1.5e-7 (half of it in Phi, about an fp32 rounding of 1), far below half an fp16 step of
// any output and no more than the rounding of the fp32 column sums of the gradients.
// One path for all arguments, for warps whose epilogue shares its issue slots with the decoding;
// GELU costs 758 us against 753 without (2048 x 28672 x 8192).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = fabsf(z) * kSqrtHalf;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  e = __expf(-x * x);
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float tail = 0.5f * p * t * e;  // Phi(-|z|)
  return z < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float act_forward(int act, float z) {
  switch (act) {
    case QL_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case QL_ACT_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case QL_ACT_GELU_TANH:
      return z * sigmoid(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
    case QL_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

// Value and derivative.
__device__ __forceinline__ void act_both(int act, float z, float& f, float& df) {
  switch (act) {
    case QL_ACT_RELU:
      f = z < 0.f ? 0.f : z;
      df = z > 0.f ? 1.f : 0.f;
      return;
    case QL_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      f = z * cdf;
      df = fmaf(z * kInvSqrt2Pi, e, cdf);
      return;
    }
    case QL_ACT_GELU_TANH: {
      const float s = sigmoid(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
      f = z * s;
      df = fmaf(z * s * (1.f - s), 2.f * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z), s);
      return;
    }
    case QL_ACT_SILU: {
      const float s = sigmoid(z);
      f = z * s;
      df = s * fmaf(z, 1.f - s, 1.f);
      return;
    }
    default:
      f = z;
      df = 1.f;
      return;
  }
}

}  // namespace qact
