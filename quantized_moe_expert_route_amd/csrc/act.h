// The activations of the 16-bit layers and their slopes, in binary32.
#pragma once

#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>

#include <type_traits>

#include "qmoe.h"

namespace qmoe {

// 1 / (1 + exp(-z)): 0 and 1 in the limits, NaN for NaN. exp2 and the reciprocal
// are the hardware's, within a unit in the last place each.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// Arguments of -inf and +inf (saved in fp16, every sum past 65504 is one) take the limits:
// z is bounded by the largest number where it multiplies what is 0 there. NaN stays NaN
// through the other factor, for min and max drop it.
__device__ __forceinline__ float above(float z) { return fmaxf(z, -FLT_MAX); }
__device__ __forceinline__ float within(float z) { return fminf(above(z), FLT_MAX); }

// u of gelu_tanh = z (1 + tanh u) / 2 = z sigmoid(2 u).
__device__ __forceinline__ float gelu_tanh_2u(float z) { return z * (1.5957691216057308f + 0.0713548162726009f * z * z); }

// The normal distribution function Phi(z), and exp(-z^2 / 2) beside it: Phi(-x) = exp(-x^2 / 2)
// R(x), x >= 0, with R a polynomial in t = 1 / (1 + 0.3 x) without a constant (R falls as 1 / x),
// fitted to erfcx(x / sqrt 2) / 2 over [0, 14.5], where Phi leaves binary32's range: least
// largest relative error, 1.6e-7 = 2.7 U (U = 2^-24). With the arithmetic the lower tail, which
// gelu multiplies by z, is off by (12 + 2 z^2) U of itself (z^2 / 2 as an exponent is rounded;
// z's own rounding moves the tail by z^2 U). (A form that is exact in absolute terms only, Abramowitz and
// Stegun 7.1.26, lost 0.16 % at z = -5 and took the same time; erff, which branches by ranges, cost
// 4096 x 6144 x 6144 45 us of 250 more.)
__device__ __forceinline__ float normal_cdf(float z, float& density) {
  const float x = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3f * x);
  density = __builtin_amdgcn_exp2f(-0.72134752044448170f * (x * x));
  const float p = t * (0.119632013f + t * (0.120712139f + t * (0.100175962f + t * (0.127691716f + t * (-0.0520339124f +
                  t * (0.204556659f + t * (-0.156158388f + t * 0.0354237258f)))))));
  const float tail = p * density;
  return z < 0.f ? tail : 1.0f - tail;
}

// act(z); ACT known when compiling: with the choice inside, every element branches.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;
  else if constexpr (ACT == MOE_ACT_SILU) return above(z) * sigmoid(z);
  else if constexpr (ACT == MOE_ACT_GELU) {
    float density;
    return above(z) * normal_cdf(z, density);
  } else if constexpr (ACT == MOE_ACT_GELU_TANH) return above(z) * sigmoid(gelu_tanh_2u(z));
  else return z;
}

// act'(z), and act(z) beside it.
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float& value) {
  if constexpr (ACT == MOE_ACT_RELU) {
    value = z < 0.f ? 0.f : z;
    return z <= 0.f ? 0.f : z != z ? z : 1.f;
  } else if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid(z);
    value = above(z) * s;
    return s * (1.f + within(z) * (1.f - s));
  } else if constexpr (ACT == MOE_ACT_GELU) {
    float density;
    const float cdf = normal_cdf(z, density);
    value = above(z) * cdf;
    return cdf + within(z) * 0.3989422804014327f * density;
  } else if constexpr (ACT == MOE_ACT_GELU_TANH) {
    // past 16 in magnitude sigmoid(2u) is 0 or 1 in binary32 and the second term
    // is 0: bounded there, so that it is not infinity times zero
    const float c = z < -16.f ? -16.f : z > 16.f ? 16.f : z;
    const float s = sigmoid(gelu_tanh_2u(c));
    value = above(z) * sigmoid(gelu_tanh_2u(z));
    return s + c * s * (1.f - s) * (1.5957691216057308f + 0.2140644488178027f * c * c);
  } else {
    value = z;
    return 1.f;
  }
}

// f with the activation's number as a constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case MOE_ACT_RELU: return f(std::integral_constant<int, MOE_ACT_RELU>{});
    case MOE_ACT_SILU: return f(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU: return f(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH: return f(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    default: return f(std::integral_constant<int, MOE_ACT_NONE>{});
  }
}

}  // namespace qmoe
