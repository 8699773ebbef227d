// fp4_act.cuh -- activation functions and their derivatives in FP32.
//
//   RELU       max(x, 0)                        slope 1 where x > 0, else 0
//   SILU       x s(x)                           s + x s (1 - s),  s(x) = 1 / (1 + e^-x)
//   GELU       x Phi(x)                         Phi(x) + x phi(x)
//   GELU_TANH  x s(2 c (x + a x^3))             s + x s (1 - s) 2 c (1 + 3 a x^2)
//              c = sqrt(2 / pi), a = 0.044715: (1 + tanh y) / 2 = s(2y), so the tanh form needs
//              one exponential, and no difference of nearly equal numbers for x << 0
//
// s is one exponential and one reciprocal of the special-function unit (relative errors of
// about 2^-21 and 2^-23, far below the half step 2^-9 of a BF16 result).  For x -> -inf,
// 1 + e^-x overflows to inf and s is 0, as it should be.
#pragma once

#include "fp4_ops.h"

namespace fp4 {

__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGeluA = 0.044715f;
constexpr float kGelu2C = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActRelu) return fmaxf(x, 0.0f);
  else if constexpr (ACT == kActSilu) return x * sigmoid_f(x);
  else if constexpr (ACT == kActGelu) return 0.5f * x * (1.0f + erff(x * kSqrtHalf));
  else if constexpr (ACT == kActGeluTanh) return x * sigmoid_f(kGelu2C * x * (1.0f + kGeluA * x * x));
  else return x;
}

// value and slope together (they share the exponential)
template <int ACT>
__device__ __forceinline__ float act_slope(float x, float& value) {
  if constexpr (ACT == kActRelu) {
    value = fmaxf(x, 0.0f);
    return x > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float s = sigmoid_f(x);
    value = x * s;
    return s * (1.0f + x * (1.0f - s));
  } else if constexpr (ACT == kActGelu) {
    const float phi = 0.5f * (1.0f + erff(x * kSqrtHalf));
    value = x * phi;
    return phi + x * kInvSqrt2Pi * __expf(-0.5f * x * x);
  } else if constexpr (ACT == kActGeluTanh) {
    // beyond |x| = 64 the sigmoid is 0 or 1: clamping keeps 0 times a large product from
    // becoming 0 times infinity
    const float c = fminf(fmaxf(x, -64.0f), 64.0f), c2 = c * c;
    const float s = sigmoid_f(kGelu2C * c * (1.0f + kGeluA * c2));
    value = x * s;
    return s * (1.0f + c * (1.0f - s) * kGelu2C * (1.0f + 3.0f * kGeluA * c2));
  } else {
    value = x;
    return 1.0f;
  }
}

// Calls f with the activation as a compile-time constant.
template <int A>
struct ActTag {
  static constexpr int value = A;
};
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(ActTag<kActRelu>{}); break;
    case kActSilu: f(ActTag<kActSilu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    default: f(ActTag<kActNone>{}); break;
  }
}

}  // namespace fp4
