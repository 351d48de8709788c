// linear_epi.cuh — the activations of the matrix products' epilogues and of their
// gradients, in fp32. Forward activations work on two values at a time: their multiplies
// and adds are packed (f32x2), which leaves the two special-function instructions per
// value (an exponential and a reciprocal, 16 per SM and cycle) as what bounds them; a
// 1024-long product's epilogue has a quarter of a cycle per output and SM in all.
#pragma once
#include <cuda_bf16.h>
#include <type_traits>

#include "block_ops.h"
#include "sm100.cuh"

namespace infini {

constexpr float kLog2e = 1.4426950408889634f;

// 1 / x to about one unit in the last place; 0 for an infinite x.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + 2^t), elementwise: 0 where 2^t overflows.
__device__ __forceinline__ uint64_t sigmoid_exp2(uint64_t t) {
  float a, b;
  f2unpack(t, a, b);
  f2unpack(add2(f2pack(ex2_approx(a), ex2_approx(b)), both(1.f)), a, b);
  return f2pack(rcp_approx(a), rcp_approx(b));
}

// Phi(-az) of the normal distribution for az >= 0, and e = exp(-az^2 / 2): e t (c0 + c1 t + ...
// + c7 t^7) with t = 1 / (1 + 0.306 az). The coefficients are a fit of this file's own, by
// reweighted least squares against Phi(-az) / e over 0 <= az <= 14.5 for the least largest
// relative error, 1.1e-7 (3.6e-7 evaluated in fp32). It is the relative error that counts:
// for v < 0 gelu is -|v| Phi(-|v|) with nothing larger beside it. What e adds is az^2 2^-22
// relative, 2^-16 at az = 8, far below the bf16 rounding of the result.
__device__ __forceinline__ uint64_t normal_tail(uint64_t az, uint64_t& e) {
  const uint64_t d = fma2(az, both(0.306f), both(1.f));
  const uint64_t x = mul2(mul2(az, az), both(-0.5f * kLog2e));
  float a, b;
  f2unpack(d, a, b);
  const uint64_t t = f2pack(rcp_approx(a), rcp_approx(b));
  f2unpack(x, a, b);
  e = f2pack(ex2_approx(a), ex2_approx(b));
  uint64_t q = fma2(t, both(0.0365375690f), both(-0.150698826f));
  q = fma2(t, q, both(0.179383233f));
  q = fma2(t, q, both(-0.0330344550f));
  q = fma2(t, q, both(0.118628532f));
  q = fma2(t, q, both(0.104367673f));
  q = fma2(t, q, both(0.122772224f));
  q = fma2(t, q, both(0.122044101f));
  return mul2(mul2(t, q), e);
}

// relu(v) = max(v, 0) (a NaN stays one); silu(v) = v / (1 + e^-v); gelu(v) = v Phi(v) =
// max(v, 0) - |v| Phi(-|v|), Phi the normal distribution (beyond |v| = 100 the second term
// is 0); its tanh form v (1 + tanh u) / 2, u = sqrt(2 / pi) (v + 0.044715 v^3), equals
// v / (1 + e^-2u), which costs no more than silu and has no cancellation for v < 0.
template <int ACT>
__device__ __forceinline__ void act_pair(float& a, float& b) {
  const uint64_t v = f2pack(a, b);
  if constexpr (ACT == kActRelu) {
    a = a < 0.f ? 0.f : a;
    b = b < 0.f ? 0.f : b;
  } else if constexpr (ACT == kActSilu) {
    f2unpack(mul2(v, sigmoid_exp2(mul2(v, both(-kLog2e)))), a, b);
  } else if constexpr (ACT == kActGeluTanh) {
    const uint64_t p =
        fma2(mul2(v, v), both(-0.071354816f * kLog2e), both(-1.5957691f * kLog2e));
    f2unpack(mul2(v, sigmoid_exp2(mul2(v, p))), a, b);
  } else if constexpr (ACT == kActGelu) {
    uint64_t e;
    const uint64_t az = f2pack(fminf(fabsf(a), 100.f), fminf(fabsf(b), 100.f));
    const uint64_t neg = mul2(az, both(-1.f));
    const uint64_t relu = f2pack(a < 0.f ? 0.f : a, b < 0.f ? 0.f : b);
    f2unpack(fma2(neg, normal_tail(az, e), relu), a, b);
  }
}

// Derivatives. relu'(0) = 0. silu' = s (1 + v (1 - s)), s = 1 / (1 + e^-v); gelu' = Phi(v) +
// v phi(v), Phi(v) = 1 - Phi(-v); tanh form with s = 1 / (1 + e^-2u): s + v s (1 - s) 2u'.
template <int ACT>
__device__ __forceinline__ void act_deriv_pair(float& a, float& b) {
  const uint64_t v = f2pack(a, b), one = both(1.f), minus = both(-1.f);
  if constexpr (ACT == kActRelu) {
    a = a <= 0.f ? 0.f : 1.f;
    b = b <= 0.f ? 0.f : 1.f;
  } else if constexpr (ACT == kActSilu) {
    const uint64_t s = sigmoid_exp2(mul2(v, both(-kLog2e)));
    f2unpack(mul2(s, fma2(v, fma2(s, minus, one), one)), a, b);
  } else if constexpr (ACT == kActGeluTanh) {
    // s is 0 or 1 long before v^2 overflows; kept finite, so that 0 times du stays 0
    const uint64_t q = f2pack(fminf(a * a, 1e30f), fminf(b * b, 1e30f));
    const uint64_t p = fma2(q, both(-0.071354816f * kLog2e), both(-1.5957691f * kLog2e));
    const uint64_t s = sigmoid_exp2(mul2(v, p));
    const uint64_t du = fma2(q, both(0.21406445f), both(1.5957691f));
    f2unpack(fma2(mul2(mul2(v, s), fma2(s, minus, one)), du, s), a, b);
  } else if constexpr (ACT == kActGelu) {
    uint64_t e;
    const uint64_t t = normal_tail(f2pack(fminf(fabsf(a), 100.f), fminf(fabsf(b), 100.f)), e);
    float ta, tb;
    f2unpack(t, ta, tb);
    const uint64_t cdf = f2pack(a < 0.f ? ta : 1.f - ta, b < 0.f ? tb : 1.f - tb);
    f2unpack(fma2(mul2(v, both(0.39894228f)), e, cdf), a, b);
  } else {
    a = b = 1.f;
  }
}

// f applied with the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    default: break;
  }
}

}  // namespace infini
