// The gated pair's activations and their derivatives, in float32.
#pragma once

#include "../../include/lq_gated.h"
#include "lq_device.h"

namespace lq {

// 1 / (1 + e^-x): the hardware's exponential and reciprocal; relative error
// about |x| 2^-24 + 2^-22 (the product x log2 e is rounded before it is raised).
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.442695040888963f));
}

struct ActPair {
  float value, slope;
};
// silu: x s with s = sigmoid(x); slope s (1 + x (1 - s)).
// gelu: x Phi(x), Phi by erfc so that its lower tail keeps its digits; slope Phi + x phi(x).
// gelu_tanh: x s with s = sigmoid(2 y), y = c (x + b x^3), the same as x (1 + tanh y) / 2;
// slope s + x s (1 - s) 2 y'. From |x| = 16 on s (1 - s) is 0: x is multiplied by it first,
// and x^2 in y' ends at 1024, so that no infinity of large finite x meets it (an infinite x gives NaN).
template <int ACT>
__device__ __forceinline__ ActPair act_pair(float x) {
  if (ACT == LQ_SILU) {
    const float s = sigmoid(x);
    return {x * s, s * __builtin_fmaf(x, 1.0f - s, 1.0f)};
  }
  if (ACT == LQ_GELU) {
    const float phi = 0.5f * erfcf(x * -0.7071067811865476f);
    const float pdf = 0.3989422804014327f * __builtin_amdgcn_exp2f(x * x * -0.7213475204444817f);
    return {x * phi, __builtin_fmaf(x, pdf, phi)};
  }
  const float c = 0.7978845608028654f, b = 0.044715f, x2 = x * x;
  const float s = sigmoid(2.0f * c * x * __builtin_fmaf(b, x2, 1.0f));
  const float slope = 2.0f * c * __builtin_fmaf(3.0f * b, fminf(x2, 1024.0f), 1.0f);
  return {x * s, __builtin_fmaf(x * (s * (1.0f - s)), slope, s)};
}
template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  return act_pair<ACT>(x).value;
}

}  // namespace lq
