// Activation functions of the fused linear layers and their derivatives, on fp32 values.
//
//   relu       max(z, 0)                        derivative: 1 for z > 0, else 0
//   gelu       z Phi(z), Phi the normal CDF     Phi(z) + z phi(z)
//   gelu_tanh  z sigma(2 v), v = sqrt(2 / pi) (z + 0.044715 z^3)  (= z (1 + tanh v) / 2, in the
//              form that does not cancel for small or very negative v)
//   silu       z sigma(z)                       sigma(z) (1 + z (1 - sigma(z)))
//
// Values (the epilogues): the fast exponential, off by 2 + |1.173 x| ulp, and division, 2 ulp.
// Relative to the value that is at most 2^-15 wherever an fp16 output is not zero (the exponent's
// own rounding at x = 30 included, which a gated product with a large factor still shows), a
// sixteenth of half an fp16 step, at every z: no value is formed by a difference.
// Gradients: the same where they are rounded to fp16 (FAST), expf and true divisions where they are
// summed in fp32.
#pragma once
#include "qlinear.h"

namespace qact {

__host__ __device__ constexpr bool act_ok(int act) { return act >= QL_ACT_NONE && act <= QL_ACT_SILU; }

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + e^-x): 0 and 1 at the far ends.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// sigma(x) and 1 - sigma(x), neither by a difference.
template <bool FAST>
__device__ __forceinline__ void sigmoid_both(float x, float& s, float& c) {
  const float e = FAST ? __expf(-fabsf(x)) : expf(-fabsf(x));
  const float r = FAST ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e), er = e * r;
  s = x < 0.f ? er : r;
  c = x < 0.f ? r : er;
}

// Phi(z) and e^(-z^2 / 2), without branches.  Phi(-|z|) = erfcx(x) e^(-x^2) / 2, x = |z| / sqrt 2,
// where erfcx(x) = e^(x^2) erfc(x) falls smoothly like 1 / x: t q(t), t = 1 / (1 + 0.6 x), q the
// polynomial of degree 7 with the least relative error over 0 <= x <= 12 (fitted by reweighted
// least squares on 4000 Chebyshev points; coefficients halved here).  Relative error 3.1e-7, in
// fp32 with an exact exponential 6e-7 for |z| <= 2 and 1.5e-6 for |z| <= 8: a tail keeps its
// digits.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float d = fmaf(0.6f * kSqrtHalf, fabsf(z), 1.f), x2 = (-0.5f * z) * z;
  const float t = FAST ? __fdividef(1.f, d) : 1.f / d;
  e = FAST ? __expf(x2) : expf(x2);
  float q = fmaf(-0.0460444614f, t, 0.205987081f);
  q = fmaf(q, t, -0.322253346f);
  q = fmaf(q, t, 0.141909704f);
  q = fmaf(q, t, 0.0366919786f);
  q = fmaf(q, t, 0.145804957f);
  q = fmaf(q, t, 0.16862385f);
  q = fmaf(q, t, 0.169280097f);
  const float tail = q * t * e;  // Phi(-|z|)
  return z < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float act_forward(int act, float z) {
  switch (act) {
    case QL_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case QL_ACT_GELU: {
      float e;
      return z * normal_cdf<true>(z, e);
    }
    case QL_ACT_GELU_TANH:
      return z * sigmoid(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
    case QL_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

// Value and derivative.
template <bool FAST>
__device__ __forceinline__ void act_both(int act, float z, float& f, float& df) {
  float s, c;
  switch (act) {
    case QL_ACT_RELU:
      f = z < 0.f ? 0.f : z;
      df = z > 0.f ? 1.f : 0.f;
      return;
    case QL_ACT_GELU: {
      float e;
      const float cdf = normal_cdf<FAST>(z, e);
      f = z * cdf;
      df = fmaf(z * kInvSqrt2Pi, e, cdf);
      return;
    }
    case QL_ACT_GELU_TANH: {
      sigmoid_both<FAST>(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z), s, c);
      f = z * s;
      // (f c is 0 long before 10^4; the square of a bf16 z would overflow and make that a NaN)
      const float a = fminf(fabsf(z), 1e4f);
      df = fmaf(f * c, 2.f * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * a * a), s);
      return;
    }
    case QL_ACT_SILU:
      sigmoid_both<FAST>(z, s, c);
      f = z * s;
      df = fmaf(f, c, s);
      return;
    default:
      f = z;
      df = 1.f;
      return;
  }
}

}  // namespace qact
