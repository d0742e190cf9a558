// dg_act.h -- activations of the linear-layer epilogue and their derivatives
// (device code), in fp32.
//
//   relu       max(x, 0)
//   gelu       x Phi(x),  Phi the normal distribution function
//   gelu_tanh  x/2 (1 + tanh u) = x / (1 + e^(-2u)),  u = sqrt(2/pi) (x + 0.044715 x^3)
//   silu       x / (1 + e^-x)
//
// Phi comes from the published five-term approximation of the error function
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26:
// erfc(z) = t (a1 + t (a2 + ...)) e^(-z^2), t = 1 / (1 + p z), z >= 0, error
// below 1.5e-7): one exponential, one reciprocal and a handful of FMAs, where
// the library's erff takes some 40 instructions -- at 128 outputs per lane
// that would be a tenth of a K = 2048 tile's time.  For x < 0 the result is
// x/2 erfc(|x| / sqrt 2) directly, without a subtraction from one.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/dg.h"

namespace dg {
namespace act {

// e^x through the base-2 exponential unit (the argument's rounding costs
// |x| 2^-24 of relative error: 1e-6 at |x| = 16).
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-x)); }

// Phi(x), and e^(-x^2 / 2) for the derivative.
__device__ __forceinline__ float phi(float x, float& e) {
  const float z = fabsf(x) * 0.70710678118654752f;
  e = exp_fast(-z * z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, z, 1.f));
  float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  p = __builtin_fmaf(p, t, 1.421413741f);
  p = __builtin_fmaf(p, t, -0.284496736f);
  p = __builtin_fmaf(p, t, 0.254829592f);
  const float half_erfc = 0.5f * p * t * e;
  return x < 0.f ? half_erfc : 1.f - half_erfc;
}

__device__ __forceinline__ float tanh_arg2(float x) {  // 2u of gelu_tanh
  return 1.59576912160573071f * __builtin_fmaf(0.044715f * x * x, x, x);
}

template <int A>
__device__ __forceinline__ float apply_one(float x) {
  if constexpr (A == DG_ACT_RELU) return x > 0.f || x != x ? x : 0.f;  // NaN stays NaN
  if constexpr (A == DG_ACT_GELU) {
    float e;
    return x * phi(x, e);
  }
  if constexpr (A == DG_ACT_GELU_TANH) return x * sigmoid(tanh_arg2(x));
  if constexpr (A == DG_ACT_SILU) return x * sigmoid(x);
  return x;
}

// The activation `a` (wave-uniform) of N values: one branch for all of them.
template <int N, class V>
__device__ __forceinline__ void apply(V& v, int a) {
#define DG_APPLY(A)                                            \
  case A:                                                      \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = apply_one<A>(v[i]); \
    break;
  switch (a) {
    DG_APPLY(DG_ACT_RELU)
    DG_APPLY(DG_ACT_GELU)
    DG_APPLY(DG_ACT_GELU_TANH)
    DG_APPLY(DG_ACT_SILU)
    default: break;
  }
#undef DG_APPLY
}

// The derivative (relu: 0 at 0).
template <int A>
__device__ __forceinline__ float grad_one(float x) {
  if constexpr (A == DG_ACT_RELU) return x > 0.f ? 1.f : 0.f;
  if constexpr (A == DG_ACT_GELU) {
    float e;
    const float p = phi(x, e);
    return __builtin_fmaf(x * 0.39894228040143268f, e, p);
  }
  if constexpr (A == DG_ACT_GELU_TANH) {
    // (beyond |x| = 11 s is 0 or 1 in fp32 and so is the slope; |x| <= 16 keeps x du2,
    // which would overflow from 1e13, finite beside the 0 of s (1 - s); NaN stays)
    x = fabsf(x) > 16.f ? __builtin_copysignf(16.f, x) : x;
    const float s = sigmoid(tanh_arg2(x));
    const float du2 = 1.59576912160573071f * __builtin_fmaf(0.134145f * x, x, 1.f);
    return __builtin_fmaf(x * du2, s * (1.f - s), s);
  }
  if constexpr (A == DG_ACT_SILU) {
    const float s = sigmoid(x);
    return __builtin_fmaf(x, s * (1.f - s), s);
  }
  return 1.f;
}

// d[i] *= activation'(x[i]) for N values.
template <int N>
__device__ __forceinline__ void times_grad(float* d, const float* x, int a) {
#define DG_GRAD(A)                                             \
  case A:                                                      \
    _Pragma("unroll") for (int i = 0; i < N; ++i) d[i] *= grad_one<A>(x[i]); \
    break;
  switch (a) {
    DG_GRAD(DG_ACT_RELU)
    DG_GRAD(DG_ACT_GELU)
    DG_GRAD(DG_ACT_GELU_TANH)
    DG_GRAD(DG_ACT_SILU)
    default: break;
  }
#undef DG_GRAD
}

}  // namespace act
}  // namespace dg
