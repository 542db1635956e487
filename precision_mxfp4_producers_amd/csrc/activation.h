// The activations of the products' epilogues and their derivatives.
#pragma once

#include "../../include/mxfp4.h"
#include "mx_device.h"

namespace mx {

// 2^x by the hardware (1 ulp).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kTanhC = -2.30220818f;                   // -2 sqrt(2/pi) log2(e)
constexpr float kTanhA = 0.044715f;

// Normal distribution function at -a, a >= 0, as 2^P(a): P is a weighted
// least-squares fit of log2(erfc(a / sqrt 2) / 2), the weights sharpened until
// the largest error of the function and of a times it was least.  In fp32
// arithmetic both are within 2.9e-7, and the function within 4e-4 of itself up to
// a = 4.5 (a bf16 rounding is up to 4e-3); from 16 on it is 0.  A fit of degree 9 in
// 1 / (1 + c a), with its reciprocal and one multiplication more, made the
// epilogue of 8192 x 14336 16 us longer at no gain in the rounded result.
__device__ __forceinline__ float normal_tail(float a) {
  float p = -0x1.b4df74p-21f;
  p = __builtin_fmaf(p, a, 0x1.51375ap-15f);
  p = __builtin_fmaf(p, a, -0x1.986106p-11f);
  p = __builtin_fmaf(p, a, 0x1.072842p-7f);
  p = __builtin_fmaf(p, a, -0x1.b43ac0p-5f);
  p = __builtin_fmaf(p, a, -0x1.d5f300p-2f);
  p = __builtin_fmaf(p, a, -0x1.26b128p+0f);
  return exp2_hw(__builtin_fmaf(p, a, -0x1.ffffe8p-1f));
}

__device__ __forceinline__ float sigmoid_of_exponent(float e) {   // 1 / (1 + 2^e)
  return __builtin_amdgcn_rcpf(__fadd_rn(1.0f, exp2_hw(e)));
}

// z times a factor that is 0 far below 0: at minus infinity their limit 0
// (a NaN comes with the factor).
__device__ __forceinline__ float times_gate(float z, float gate) { return __fmul_rn(fmaxf(z, -128.0f), gate); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == FP4_ACT_RELU) return z <= 0.0f ? 0.0f : z;
  if constexpr (ACT == FP4_ACT_GELU) {
    // z for positive z, less |z| times the tail on both sides (which is 0 from 16
    // on; a NaN comes with the tail)
    return __builtin_fmaf(-fminf(fabsf(z), 16.0f), normal_tail(fabsf(z)), fmaxf(z, 0.0f));
  }
  if constexpr (ACT == FP4_ACT_GELU_TANH)
    return times_gate(z, sigmoid_of_exponent(__fmul_rn(kTanhC, __builtin_fmaf(__fmul_rn(__fmul_rn(z, z), z), kTanhA, z))));
  if constexpr (ACT == FP4_ACT_SILU) return times_gate(z, sigmoid_of_exponent(__fmul_rn(-kLog2e, z)));
  return z;
}

// The derivative; beyond |z| = 128 all are 0 or 1 in fp32, and taken at 128.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == FP4_ACT_NONE) return 1.0f;
  if constexpr (ACT == FP4_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  const float x = __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f);
  float d = 1.0f;
  if constexpr (ACT == FP4_ACT_GELU) {
    const float q = normal_tail(fabsf(x));
    const float density = __fmul_rn(0.39894228f, exp2_hw(__fmul_rn(__fmul_rn(x, x), -0.5f * kLog2e)));
    d = __builtin_fmaf(x, density, x < 0.0f ? q : __fsub_rn(1.0f, q));
  } else if constexpr (ACT == FP4_ACT_GELU_TANH) {
    const float xx = __fmul_rn(x, x);
    const float s = sigmoid_of_exponent(__fmul_rn(kTanhC, __builtin_fmaf(__fmul_rn(xx, x), kTanhA, x)));
    const float inner = __builtin_fmaf(xx, 1.5957691f * 3.0f * kTanhA, 1.5957691f);   // 2 sqrt(2/pi) (1 + 3 A x^2)
    d = __builtin_fmaf(__fmul_rn(__fmul_rn(x, s), __fsub_rn(1.0f, s)), inner, s);
  } else if constexpr (ACT == FP4_ACT_SILU) {
    const float s = sigmoid_of_exponent(__fmul_rn(-kLog2e, x));
    d = __fmul_rn(s, __builtin_fmaf(x, __fsub_rn(1.0f, s), 1.0f));
  }
  return z == z ? d : z;
}

// f(integral_constant) with the activation as a compile-time value; one
// wave-uniform branch.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case FP4_ACT_RELU: return f(std::integral_constant<int, FP4_ACT_RELU>{});
    case FP4_ACT_GELU: return f(std::integral_constant<int, FP4_ACT_GELU>{});
    case FP4_ACT_GELU_TANH: return f(std::integral_constant<int, FP4_ACT_GELU_TANH>{});
    case FP4_ACT_SILU: return f(std::integral_constant<int, FP4_ACT_SILU>{});
    default: return f(std::integral_constant<int, FP4_ACT_NONE>{});
  }
}

}  // namespace mx
