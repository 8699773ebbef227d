// fp4_act.cuh -- activation functions and their derivatives in FP32.
//
//   RELU       max(x, 0), NaN for a NaN         slope 1 where x > 0, else 0
//   SILU       x s(x)                           s + x s (1 - s),  s(x) = 1 / (1 + e^-x)
//   GELU       x Phi(x)                         Phi(x) + x phi(x)
//   GELU_TANH  x s(2 c (x + a x^3))             s + x s (1 - s) 2 c (1 + 3 a x^2)
//              c = sqrt(2 / pi), a = 0.044715: (1 + tanh y) / 2 = s(2y), so the tanh form needs
//              one exponential, and no difference of nearly equal numbers for x << 0
//
// s is one exponential and one reciprocal of the special-function unit (relative errors of
// about 2^-21 and 2^-23, far below the half step 2^-9 of a BF16 result), both with subnormal
// results flushed to 0, which saves their scaling steps.  For x -> -inf, 1 + e^-x overflows to
// inf and s is 0, as it should be.
#pragma once

#include "fp4_ops.h"

namespace fp4 {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_sfu(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_sfu(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// s(x) from y = -x log2(e)
__device__ __forceinline__ float sigmoid_from(float y) { return rcp_sfu(1.0f + exp2_sfu(y)); }
__device__ __forceinline__ float sigmoid_f(float x) { return sigmoid_from(x * -kLog2e); }

constexpr float kGeluA = 0.044715f;
constexpr float kGelu2C = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// Phi(x), and e^(-x^2/2) for its derivative: erfc(z) = e^(-z^2) P(t), t = 1 / (1 + 0.3275911 z),
// z = |x| / sqrt(2) >= 0, the rational approximation 7.1.26 of Abramowitz and Stegun's Handbook
// of Mathematical Functions (error at most 1.5e-7; x Phi(x) / x is within 3.4e-7 over [-40, 40] in
// all, 0.2% of Phi itself at x = -5).  Half the instructions of erff, no branch, and no 1 + erf
// of nearly -1 for x << 0.
__device__ __forceinline__ float normal_cdf(float x, float& e) {
  const float z = fabsf(x) * kSqrtHalf;
  const float t = rcp_sfu(fmaf(0.3275911f, z, 1.0f));
  e = exp2_sfu(z * z * -kLog2e);
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  const float half = 0.5f * p * t * e;
  return x >= 0.0f ? 1.0f - half : half;
}

// (fmaxf would turn a NaN into 0)
__device__ __forceinline__ float relu_f(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActRelu) return relu_f(x);
  else if constexpr (ACT == kActSilu) return x * sigmoid_f(x);
  else if constexpr (ACT == kActGelu) { float e; return x * normal_cdf(x, e); }
  else if constexpr (ACT == kActGeluTanh) return x * sigmoid_from(x * fmaf(x * x, -kLog2e * kGelu2C * kGeluA, -kLog2e * kGelu2C));
  else return x;
}

// value and slope together (they share the exponential)
template <int ACT>
__device__ __forceinline__ float act_slope(float x, float& value) {
  if constexpr (ACT == kActRelu) {
    value = relu_f(x);
    return x > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float s = sigmoid_f(x);
    value = x * s;
    return s * (1.0f + x * (1.0f - s));
  } else if constexpr (ACT == kActGelu) {
    float e;
    const float phi = normal_cdf(x, e);
    value = x * phi;
    return phi + x * kInvSqrt2Pi * e;
  } else if constexpr (ACT == kActGeluTanh) {
    // beyond |x| = 64 the sigmoid is 0 or 1: clamping keeps 0 times a large product from
    // becoming 0 times infinity
    const float c = fminf(fmaxf(x, -64.0f), 64.0f), c2 = c * c;
    const float s = sigmoid_f(kGelu2C * c * (1.0f + kGeluA * c2));
    value = x * s;
    return fmaf(0.0f, x, s * (1.0f + c * (1.0f - s) * kGelu2C * (1.0f + 3.0f * kGeluA * c2)));  // a NaN stays one
  } else {
    value = x;
    return 1.0f;
  }
}

// Two values at once: the paired FP32 instructions do the arithmetic around the special
// functions, which take one value each.
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }
template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 x) {
  if constexpr (ACT == kActSilu || ACT == kActGeluTanh) {
    float2 y;
    if constexpr (ACT == kActSilu) y = __fmul2_rn(x, pair(-kLog2e));
    else y = __fmul2_rn(x, __ffma2_rn(__fmul2_rn(x, x), pair(-kLog2e * kGelu2C * kGeluA), pair(-kLog2e * kGelu2C)));
    const float2 d = __fadd2_rn(make_float2(exp2_sfu(y.x), exp2_sfu(y.y)), pair(1.0f));
    return __fmul2_rn(x, make_float2(rcp_sfu(d.x), rcp_sfu(d.y)));
  } else if constexpr (ACT == kActGelu) {  // as normal_cdf
    const float2 z = make_float2(fabsf(x.x), fabsf(x.y));
    const float2 d = __ffma2_rn(z, pair(0.3275911f * kSqrtHalf), pair(1.0f));
    const float2 t = make_float2(rcp_sfu(d.x), rcp_sfu(d.y));
    const float2 y = __fmul2_rn(__fmul2_rn(x, x), pair(-0.5f * kLog2e));
    const float2 e = make_float2(exp2_sfu(y.x), exp2_sfu(y.y));
    float2 p = __ffma2_rn(t, pair(0.5f * 1.061405429f), pair(0.5f * -1.453152027f));
    p = __ffma2_rn(t, p, pair(0.5f * 1.421413741f));
    p = __ffma2_rn(t, p, pair(0.5f * -0.284496736f));
    p = __ffma2_rn(t, p, pair(0.5f * 0.254829592f));
    const float2 half = __fmul2_rn(__fmul2_rn(p, t), e);
    const float2 rest = __ffma2_rn(half, pair(-1.0f), pair(1.0f));
    return __fmul2_rn(x, make_float2(x.x < 0.0f ? half.x : rest.x, x.y < 0.0f ? half.y : rest.y));
  } else {
    return make_float2(act_value<ACT>(x.x), act_value<ACT>(x.y));
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
