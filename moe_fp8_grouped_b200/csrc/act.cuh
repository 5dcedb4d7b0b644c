// act.cuh -- the activations of the product epilogues and their gradients.
#pragma once

#include <cuda_runtime.h>

#include "gmm_fp8.h"

namespace gmm {

__device__ __forceinline__ float act_sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(z) of the one-input activations
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case GMM_ACT_RELU: return z > 0.0f ? z : (isnan(z) ? z : 0.0f);
    case GMM_ACT_SILU: return z / (1.0f + expf(-z));
    // 0.5 z erfc(-z / sqrt 2): no cancellation for large negative z
    case GMM_ACT_GELU: return 0.5f * z * erfcf(-0.7071067811865476f * z);
    // 0.5 z (1 + tanh(u)) = z sigmoid(2 u)
    case GMM_ACT_GELU_TANH: return z / (1.0f + expf(-2.0f * kGeluC * (z + kGeluA * z * z * z)));
    default: return z;
  }
}

// d act(z) / dz
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case GMM_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case GMM_ACT_SILU: {
      const float s = act_sigmoid(z);
      return s * (1.0f + z * (1.0f - s));
    }
    case GMM_ACT_GELU:
      return 0.5f * erfcf(-0.7071067811865476f * z) + z * (0.3989422804014327f * expf(-0.5f * z * z));
    case GMM_ACT_GELU_TANH: {
      if (fabsf(z) > 16.0f) return z > 0.0f ? 1.0f : 0.0f;  // to fp32; z^3 below stays finite
      const float s = act_sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
      return s + z * s * (1.0f - s) * (2.0f * kGeluC * (1.0f + 3.0f * kGeluA * z * z));
    }
    default: return 1.0f;
  }
}

}  // namespace gmm
