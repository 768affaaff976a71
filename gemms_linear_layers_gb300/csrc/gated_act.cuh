// gated_act.cuh -- the gate's activations and their derivatives, in FP32.
#pragma once
#include "gated.h"
#include "ptx.cuh"

namespace tg {

// 1 / (1 + e^-x): 0 and 1 at the ends (the divide gives 0 for a denominator of 2^126 or more)
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// The normal distribution's function by its upper tail, erfc(z) / 2 at z = |x| / sqrt(2), so that
// it keeps its relative accuracy where 1 + erf cancels: erfc(z) = t e^(p(t) - z^2) with
// t = 1 / (1 + z / 2) (the form of Press, Teukolsky, Vetterling and Flannery, Numerical Recipes,
// 6.2), p fitted here: the polynomial of degree 7 through ln(erfc(z) e^(z^2) / t) at Chebyshev
// points of t for z in [0, 10] (from there on the tail is below FP32's range).  Off by at most
// 1.1e-6 of the tail in FP32, beside e^(-z^2)'s own error, z^2 2^-23.  (erfcf in its place made the
// block of 1,001 rows, 576 -> 1,536 4.5 us slower than SiLU.)
__device__ __forceinline__ float tail_exponent(float t) {
  float p = -0.18845126f;
  p = fmaf(p, t, 0.75412422f);
  p = fmaf(p, t, -1.00495267f);
  p = fmaf(p, t, 0.35287324f);
  p = fmaf(p, t, -0.04086587f);
  p = fmaf(p, t, 0.39417261f);
  p = fmaf(p, t, 0.99857694f);
  return fmaf(p, t, -1.2654779f);
}
__device__ __forceinline__ float normal_cdf(float x) {
  const float z = fabsf(x) * 0.70710678118654752f, t = __fdividef(1.f, fmaf(0.5f, z, 1.f));
  const float tail = 0.5f * t * __expf(fmaf(-z, z, tail_exponent(t)));
  return x > 0.f ? 1.f - tail : tail;
}
// with e^(-x^2 / 2) beside it
__device__ __forceinline__ float normal_cdf(float x, float* bell) {
  const float z = fabsf(x) * 0.70710678118654752f, t = __fdividef(1.f, fmaf(0.5f, z, 1.f));
  *bell = __expf(-z * z);
  const float tail = 0.5f * t * __expf(tail_exponent(t)) * *bell;
  return x > 0.f ? 1.f - tail : tail;
}

// The tanh form of GELU is x s(y), s the logistic function, y = 2 sqrt(2/pi) (x + 0.044715 x^3)
constexpr float GELU_K = 1.5957691216057308f, GELU_C = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activation(float x) {
  if constexpr (ACT == ACT_SILU) return x * logistic(x);
  else if constexpr (ACT == ACT_GELU) return x * normal_cdf(x);
  else if constexpr (ACT == ACT_GELU_TANH) return x * logistic(GELU_K * fmaf(GELU_C * x * x, x, x));
  else return x < 0.f ? 0.f : x;  // not fmaxf: a value that is not a number stays one
}

template <int ACT>
__device__ __forceinline__ float activation_grad(float x, float* value) {
  if constexpr (ACT == ACT_SILU) {
    const float p = logistic(x);
    *value = x * p;
    return p * fmaf(x, 1.f - p, 1.f);
  } else if constexpr (ACT == ACT_GELU) {
    float bell;
    const float p = normal_cdf(x, &bell);
    *value = x * p;
    return fmaf(x, 0.39894228040143268f * bell, p);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float p = logistic(GELU_K * fmaf(GELU_C * x * x, x, x));
    *value = x * p;
    // beyond 12 the factor p (1 - p) is 0 in FP32, and x^2 of the largest x must not make it 0 inf
    const float z = fminf(fmaxf(x, -12.f), 12.f);
    return fmaf(z * p * (1.f - p), GELU_K * fmaf(3.f * GELU_C * z, z, 1.f), p);
  } else {
    *value = x < 0.f ? 0.f : x;
    return x > 0.f ? 1.f : 0.f;
  }
}

}  // namespace tg
