// linear_epi.cuh — the activations of the matrix products' epilogues and of their
// gradients, in fp32.
#pragma once
#include <cuda_bf16.h>

#include "block_ops.h"

namespace infini {

// relu(v) = max(v, 0) (a NaN stays one); silu(v) = v / (1 + e^-v);
// gelu(v) = v Phi(v) = v (1 + erf(v / sqrt 2)) / 2; its tanh form
// v (1 + tanh u) / 2, u = sqrt(2 / pi) (v + 0.044715 v^3), equals v / (1 + e^-2u), which
// costs one exponential and one division like silu and has no cancellation for v < 0.
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == kActRelu) return v < 0.f ? 0.f : v;
  if constexpr (ACT == kActSilu) return __fdividef(v, 1.f + __expf(-v));
  if constexpr (ACT == kActGelu) return 0.5f * v * (1.f + erff(v * 0.70710678f));
  if constexpr (ACT == kActGeluTanh) {
    const float m2u = v * fmaf(v * v, -0.071354816f, -1.5957691f);  // -2u
    return __fdividef(v, 1.f + __expf(m2u));
  }
  return v;
}

// Derivatives. relu'(0) = 0. silu' = s (1 + v (1 - s)); gelu' = Phi(v) + v phi(v); tanh
// form with s = 1 / (1 + e^-2u): s + v s (1 - s) 2u'.
template <int ACT>
__device__ __forceinline__ float act_deriv(float v) {
  if constexpr (ACT == kActRelu) return v <= 0.f ? 0.f : 1.f;
  if constexpr (ACT == kActSilu) {
    const float s = __fdividef(1.f, 1.f + __expf(-v));
    return s * fmaf(v, 1.f - s, 1.f);
  }
  if constexpr (ACT == kActGelu)
    return fmaf(v * 0.39894228f, __expf(-0.5f * v * v), 0.5f * (1.f + erff(v * 0.70710678f)));
  if constexpr (ACT == kActGeluTanh) {
    const float q = v * v;
    const float s = __fdividef(1.f, 1.f + __expf(v * fmaf(q, -0.071354816f, -1.5957691f)));
    return fmaf(v * s * (1.f - s), fmaf(q, 0.21406445f, 1.5957691f), s);
  }
  return 1.f;
}

// f applied with the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

}  // namespace infini
