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

// Square root of the normal distribution function at -a, a >= 0, as 2^P(a): 2 P is a
// minimax fit of log2(erfc(a / sqrt 2) / 2) up to a = 13.6, its tolerance a relative
// error far out and an absolute one of the function near 0.  Of degree 10, for
// values rounded to bf16, the function is within 1e-3 of itself (a bf16 rounding is up
// to 4e-3) and gelu of normal z within 1.7e-7 in the 2-norm; of degree 12 (FINE) within
// 8e-5 of itself up to 8 and 3e-4 up to 13, and gelu within 5.2e-8 (fp32's erfc:
// 3.3e-8).  The root, since the hardware's 2^x is 0 below 2^-126, where a times the
// function is still a normal number.  Even degrees with a negative last coefficient:
// far out P is minus infinity.
// 8192 x 14336 x 4096 with GELU: 300 us with a bf16 y, degree 12 instead 306; 324 with
// an fp32 one.  A fit of degree 7, off by a tenth at a = 8, took 295 and 313.
template <bool FINE>
__device__ __forceinline__ float normal_tail_root(float a) {
  float p;
  if constexpr (FINE) {
    p = __builtin_fmaf(-0x1.8b0816p-38f, a, 0x1.de93f0p-32f);
    p = __builtin_fmaf(p, a, -0x1.f62538p-27f);
    p = __builtin_fmaf(p, a, 0x1.29b9d6p-22f);
    p = __builtin_fmaf(p, a, -0x1.b1f1c6p-19f);
    p = __builtin_fmaf(p, a, 0x1.832ec6p-16f);
    p = __builtin_fmaf(p, a, -0x1.5e8292p-14f);
    p = __builtin_fmaf(p, a, -0x1.f74ef8p-14f);
    p = __builtin_fmaf(p, a, 0x1.da4802p-9f);
    p = __builtin_fmaf(p, a, -0x1.af2348p-6f);
    p = __builtin_fmaf(p, a, -0x1.d62ed6p-3f);
    p = __builtin_fmaf(p, a, -0x1.26af30p-1f);
    return exp2_hw(__builtin_fmaf(p, a, -0x1.fffffcp-2f));
  } else {
    p = __builtin_fmaf(-0x1.7cfadep-32f, a, 0x1.4f6e56p-26f);
    p = __builtin_fmaf(p, a, -0x1.ccada0p-22f);
    p = __builtin_fmaf(p, a, 0x1.1a80f4p-18f);
    p = __builtin_fmaf(p, a, -0x1.7b273ep-18f);
    p = __builtin_fmaf(p, a, -0x1.467c74p-12f);
    p = __builtin_fmaf(p, a, 0x1.fd49b4p-9f);
    p = __builtin_fmaf(p, a, -0x1.b260d2p-6f);
    p = __builtin_fmaf(p, a, -0x1.d60ad4p-3f);
    p = __builtin_fmaf(p, a, -0x1.26b050p-1f);
    return exp2_hw(__builtin_fmaf(p, a, -0x1.fffff2p-2f));
  }
}

__device__ __forceinline__ float sigmoid_of_exponent(float e) {   // 1 / (1 + 2^e)
  return __builtin_amdgcn_rcpf(__fadd_rn(1.0f, exp2_hw(e)));
}

// z times a factor that is 0 far below 0: at minus infinity their limit 0
// (a NaN comes with the factor).
__device__ __forceinline__ float times_gate(float z, float gate) { return __fmul_rn(fmaxf(z, -128.0f), gate); }

// FINE: for an fp32 result; else it is rounded to bf16.
template <int ACT, bool FINE>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == FP4_ACT_RELU) return z <= 0.0f ? 0.0f : z;
  if constexpr (ACT == FP4_ACT_GELU) {
    // z for positive z, less |z| times the tail on both sides.  |z| times the root is
    // below 1/2; the clamp, which is part of that multiplication, makes it 0 where |z|
    // is infinite (infinity times 0), and a NaN comes with the root.
    const float t = normal_tail_root<FINE>(fabsf(z));
    const float u = __builtin_amdgcn_fmed3f(__fmul_rn(fabsf(z), t), 0.0f, 1.0f);
    const float p = __int_as_float(std::max(__float_as_int(z), 0));   // max(z, 0) in one instruction
    return __builtin_fmaf(-u, t, p);
  }
  if constexpr (ACT == FP4_ACT_GELU_TANH)
    return times_gate(z, sigmoid_of_exponent(__fmul_rn(kTanhC, __builtin_fmaf(__fmul_rn(__fmul_rn(z, z), z), kTanhA, z))));
  if constexpr (ACT == FP4_ACT_SILU) return times_gate(z, sigmoid_of_exponent(__fmul_rn(-kLog2e, z)));
  return z;
}

// The derivative; beyond |z| = 128 all are 0 or 1 in fp32 (the last two are taken there).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == FP4_ACT_NONE) return 1.0f;
  if constexpr (ACT == FP4_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  if constexpr (ACT == FP4_ACT_GELU) {
    // At -|z| the tail less |z| times the density, at |z| one less that.  Both as
    // squares of their roots (the density is in range where 2^x of it is not); far out
    // the tail is a tenth of it or less, so that the shorter fit leaves 1e-4.  The clamp
    // as above: 0 where z is infinite, and a NaN comes with the roots.
    const float t = normal_tail_root<false>(fabsf(z));
    const float r = exp2_hw(__builtin_fmaf(__fmul_rn(z, z), -0.25f * kLog2e, -0.66287406f));   // log2(2 pi) / -4
    const float u = __builtin_amdgcn_fmed3f(__fmul_rn(fabsf(z), r), 0.0f, 1.0f);
    const float v = __builtin_fmaf(-u, r, __fmul_rn(t, t));
    return z < 0.0f ? v : __fsub_rn(1.0f, v);
  }
  const float x = __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f);
  float d = 1.0f;
  if constexpr (ACT == FP4_ACT_GELU_TANH) {
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
