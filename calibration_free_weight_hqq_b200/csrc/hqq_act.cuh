// hqq_act.cuh - activations of the gated products and their derivatives, in fp32.
#pragma once

#include <cuda_runtime.h>

#include "hqq_kernels.h"

namespace hqqk {

__device__ __forceinline__ float sigmoid_f32(float x) {
  return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-x)));  // exp overflow: 1 / inf = 0
}

// sqrt(2/pi) * (g + 0.044715 g^3), the argument of the tanh form of gelu.
__device__ __forceinline__ float gelu_tanh_arg(float g) {
  return 0.7978845608028654f * g * (1.0f + 0.044715f * g * g);
}

// act(g). silu: g s(g); gelu: g Phi(g), Phi through erfc (no cancellation in the lower tail);
// gelu, tanh form: g (1 + tanh y)/2 = g s(2y).
template <int ACT>
__device__ __forceinline__ float act_f32(float g) {
  if constexpr (ACT == kSilu) return g * sigmoid_f32(g);
  if constexpr (ACT == kGelu) return 0.5f * g * erfcf(-0.7071067811865476f * g);
  return g * sigmoid_f32(2.0f * gelu_tanh_arg(g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ float2 act_and_grad_f32(float g) {
  if constexpr (ACT == kSilu) {
    const float s = sigmoid_f32(g);
    return make_float2(g * s, s * (1.0f + g * (1.0f - s)));
  } else if constexpr (ACT == kGelu) {
    const float cdf = 0.5f * erfcf(-0.7071067811865476f * g);
    const float pdf = 0.3989422804014327f * __expf(-0.5f * g * g);
    return make_float2(g * cdf, cdf + g * pdf);
  } else {
    const float s = sigmoid_f32(2.0f * gelu_tanh_arg(g));
    // from |g| = 100 on s (1 - s) is 0, and neither 2 g nor g^2, which overflow, must meet it
    const float c = fminf(fmaxf(g, -100.0f), 100.0f);
    const float dy = 0.7978845608028654f * (1.0f + 0.134145f * c * c);
    return make_float2(g * s, s + 2.0f * c * s * (1.0f - s) * dy);
  }
}

}  // namespace hqqk
