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

// Epilogue of the forward kernels: the result is rounded to fp16, so the fast exponential and
// division (a few fp32 ulps) are far below half an fp16 step.  z / (1 + inf) = -0 for very
// negative z.
__device__ __forceinline__ float act_forward(int act, float z) {
  switch (act) {
    case QL_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case QL_ACT_GELU: return 0.5f * z * (1.f + erff(z * kSqrtHalf));
    case QL_ACT_GELU_TANH: {
      const float v2 = 2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z);
      return __fdividef(z, 1.f + __expf(-v2));
    }
    case QL_ACT_SILU: return __fdividef(z, 1.f + __expf(-z));
    default: return z;
  }
}

// Backward: value and derivative with the accurate functions (the bias gradient is kept in
// fp32, where the fast forms' errors would show; the kernel is bound by memory).
__device__ __forceinline__ void act_both(int act, float z, float& f, float& df) {
  switch (act) {
    case QL_ACT_RELU:
      f = z < 0.f ? 0.f : z;
      df = z > 0.f ? 1.f : 0.f;
      return;
    case QL_ACT_GELU: {
      const float cdf = 0.5f * (1.f + erff(z * kSqrtHalf));
      f = z * cdf;
      df = cdf + z * (kInvSqrt2Pi * expf(-0.5f * z * z));
      return;
    }
    case QL_ACT_GELU_TANH: {
      const float v2 = 2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z);
      const float s = 1.f / (1.f + expf(-v2));
      f = z * s;
      df = s + z * s * (1.f - s) * (2.f * kSqrt2OverPi) * (1.f + 3.f * kGeluCubic * z * z);
      return;
    }
    case QL_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-z));
      f = z * s;
      df = s * (1.f + z * (1.f - s));
      return;
    }
    default:
      f = z;
      df = 1.f;
      return;
  }
}

}  // namespace qact
