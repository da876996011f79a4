// Activation functions of the fused GEMM epilogue and the activation kernels,
// and their derivatives, in float32.
//
// The logistic function is 1 / (1 + 2^(-x log2 e)) with the hardware's exp2 and
// reciprocal (1 ulp each): the error of the rounded exponent, |x| 2^-24
// relative, matters only where the function itself is within 2^-24 |x| of its
// limit. The tanh form of GELU is x * logistic(2u), since (1 + tanh u) / 2 =
// logistic(2u): no cancellation for negative u. exp2 of a large argument is
// +Inf and its reciprocal 0, which is the limit.
//
// GELU's normal distribution function is 1 - h for x >= 0 and h below, with
// h = erfc(|x| / sqrt 2) / 2 from the rational approximation 7.1.26 of
// Abramowitz and Stegun, Handbook of Mathematical Functions: erfc(y) =
// (a1 t + ... + a5 t^5) exp(-y^2), t = 1 / (1 + p y), absolute error at most
// 1.5e-7, about a float32 rounding of the result.
#pragma once

#include <hip/hip_runtime.h>

namespace hq {

constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;

__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// 2 sqrt(2/pi) (x + 0.044715 x^3) = x (C0 + C1 x^2)
constexpr float kGeluC0 = 1.59576912f, kGeluC1 = 0.0713548163f;

// The distribution function, and exp(-x^2/2) in *g.
__device__ __forceinline__ float normal_cdf(float x, float* g) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(x), 0.3275911f * 0.707106781f, 1.0f));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  *g = __builtin_amdgcn_exp2f(x * x * -0.721347520f);
  const float h = 0.5f * t * p * *g;
  return x < 0.0f ? h : 1.0f - h;
}

// act(x)
template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActRelu) return x > 0.0f ? x : (x != x ? x : 0.0f);
  if constexpr (ACT == kActSilu) return x * logistic(x);
  if constexpr (ACT == kActGelu) {
    float g;
    return x * normal_cdf(x, &g);
  }
  if constexpr (ACT == kActGeluTanh) return x * logistic(x * fmaf(kGeluC1, x * x, kGeluC0));
  return x;
}

// act(x) and act'(x)
template <int ACT>
__device__ __forceinline__ void act_value_grad(float x, float* v, float* d) {
  if constexpr (ACT == kActRelu) {
    *v = x > 0.0f ? x : (x != x ? x : 0.0f);
    *d = x > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float p = logistic(x);
    *v = x * p;
    *d = p * fmaf(x, 1.0f - p, 1.0f);
  } else if constexpr (ACT == kActGelu) {
    float g;
    const float c = normal_cdf(x, &g);
    *v = x * c;
    *d = fmaf(x * 0.398942280f, g, c);  // 1 / sqrt(2 pi)
  } else if constexpr (ACT == kActGeluTanh) {
    const float x2 = x * x;
    const float p = logistic(x * fmaf(kGeluC1, x2, kGeluC0));
    *v = x * p;
    // derivative of the logistic's argument: 2 sqrt(2/pi) (1 + 3 * 0.044715 x^2).
    // Past |x| = 16 p is exactly 0 or 1; the clamp keeps x^3 from overflowing there.
    const float c = __builtin_amdgcn_fmed3f(x, -16.0f, 16.0f);
    *d = p * fmaf(c * fmaf(3.0f * kGeluC1, c * c, kGeluC0), 1.0f - p, 1.0f);
  } else {
    *v = x;
    *d = 1.0f;
  }
}

}  // namespace hq
