// mx_act.hpp — activations of the products with an MXFP4 operand.
#pragma once

#include "device_common.hpp"

namespace biasact {
namespace mx {

// erfc(ax) for ax >= 0 in the form and with the coefficients of erfc_f32, times
// 2^64 where `tiny` comes back true: below 2^-126 the product is formed at that
// size, so that whoever scales it back (exactly) rounds once onto the subnormal
// grid.
__device__ __forceinline__ float erfc_scaled(float ax, bool& tiny) {
#pragma clang fp contract(off)
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, ax, 1.0f));
  float p = 1.449302137e-01f;
  p = __builtin_fmaf(p, t, -6.808272004e-01f);
  p = __builtin_fmaf(p, t, 1.156733751e+00f);
  p = __builtin_fmaf(p, t, -6.962518692e-01f);
  p = __builtin_fmaf(p, t, -8.028043061e-02f);
  p = __builtin_fmaf(p, t, 1.267586369e-03f);
  p = __builtin_fmaf(p, t, 3.460279852e-02f);
  p = __builtin_fmaf(p, t, 3.866403997e-01f);
  p = __builtin_fmaf(p, t, 9.986327887e-01f);
  p = __builtin_fmaf(p, t, -1.265447974e+00f);
  const float e = __builtin_fmaf(-ax, ax, p);
  const float s = e * 1.442695041f;
  tiny = s < -126.0f;
  return t * __builtin_amdgcn_exp2f(tiny ? s + 64.0f : s);
}

// GELU whose far negative tail is formed at 2^64 times its size and scaled back
// at the very end: fp32 results below 2^-126 take one rounding onto the
// subnormal grid (gelu_f32 rounds Phi there first and then scales that error
// by z).
__device__ __forceinline__ float gelu_tail(float z) {
#pragma clang fp contract(off)
  bool tiny;
  const float r = erfc_scaled(__builtin_fabsf(z * -0.7071067812f), tiny);
  const float h = 0.5f * z;
  const float neg = tiny ? (h * r) * 0x1p-64f : h * r;
  return z > 0.0f ? h * (2.0f - (tiny ? 0.0f : r)) : neg;
}

// GELU for a result that is next rounded to fp16 or bf16:
//   gelu(z) = max(z, 0) - |z| / 2 * erfc(|z| / sqrt 2),
// the last factor as t * 2^(-z^2 log2(e) / 2 + Q(t)), t = 1 / (1 + 0.35 |z|), Q of
// degree 5 (csrc/fit_erfc.py; relative error below 2^-17, 1.3e-5 with the
// roundings).  The exponent carries 16 more and |z| / 2 that much less, so that
// results down to bf16's subnormals round once.  A positive z is bounded, so that
// infinity times zero stays out of gelu(inf) = inf; gelu(-inf) = -inf * 0 is NaN
// as in gelu_f32 and gelu_tail, and a NaN comes in through z * z.  14 instructions
// and two transcendentals for gelu_f32's 24 and two.
__device__ __forceinline__ float gelu_short(float z) {
#pragma clang fp contract(off)
  const float az = __builtin_fabsf(__builtin_fminf(z, 0x1p14f));
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(az, 0.35f, 1.0f));
  float q = 3.331241608e-01f;
  q = __builtin_fmaf(q, t, -1.050401449e+00f);
  q = __builtin_fmaf(q, t, 7.378793359e-01f);
  q = __builtin_fmaf(q, t, 3.479329050e-01f);
  q = __builtin_fmaf(q, t, 1.473684072e+00f);
  q = __builtin_fmaf(q, t, 16.0f - 1.842209578e+00f);
  const float e = __builtin_fmaf(z * z, -0.72134752f, q);
  return __builtin_fmaxf(z, 0.0f) - (az * 0x1p-17f) * (t * __builtin_amdgcn_exp2f(e));
}

// The activation for an output of type DTO: GELU to the accuracy that a 16-bit
// output keeps, and with its subnormal tail for fp32.
template <int ACT, int DTO>
__device__ __forceinline__ float act(float z, float alpha) {
  if constexpr (ACT == ACT_GELU && DTO == DT_F32) return gelu_tail(z);
  else if constexpr (ACT == ACT_GELU) return gelu_short(z);
  else return act_fn<ACT, DTO>(z, alpha);
}

}  // namespace mx
}  // namespace biasact
