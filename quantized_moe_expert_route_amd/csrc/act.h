// The activations of the 16-bit layers and their slopes, in binary32.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>

#include "qmoe.h"

namespace qmoe {

// 1 / (1 + exp(-z)): 0 and 1 in the limits, NaN for NaN.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

// u of gelu_tanh = z (1 + tanh u) / 2 = z sigmoid(2 u).
__device__ __forceinline__ float gelu_tanh_2u(float z) { return z * (1.5957691216057308f + 0.0713548162726009f * z * z); }

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;
    case MOE_ACT_SILU: return z * sigmoid(z);
    case MOE_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH: return z * sigmoid(gelu_tanh_2u(z));
    default: return z;
  }
}

// act'(z), and act(z) beside it.
__device__ __forceinline__ float act_slope(int act, float z, float& value) {
  switch (act) {
    case MOE_ACT_RELU:
      value = z < 0.f ? 0.f : z;
      return z <= 0.f ? 0.f : z != z ? z : 1.f;
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      value = z * s;
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACT_GELU: {
      const float cdf = 0.5f * (1.f + erff(z * 0.70710678118654752f));
      value = z * cdf;
      return cdf + z * 0.3989422804014327f * __expf(-0.5f * z * z);
    }
    case MOE_ACT_GELU_TANH: {
      // past 16 in magnitude sigmoid(2u) is 0 or 1 in binary32 and the second term
      // is 0: bounded there, so that it is not infinity times zero
      const float c = z < -16.f ? -16.f : z > 16.f ? 16.f : z;
      const float s = sigmoid(gelu_tanh_2u(c));
      value = z * sigmoid(gelu_tanh_2u(z));
      return s + c * s * (1.f - s) * (1.5957691216057308f + 0.2140644488178027f * c * c);
    }
    default:
      value = z;
      return 1.f;
  }
}

}  // namespace qmoe
