// The activations of the product's epilogue and their derivatives, in FP32.
// Codes as in the library's header: 0 none, 1 ReLU, 2 GELU (erf form), 3 SiLU,
// 4 GELU (tanh form).
#pragma once

#include <hip/hip_runtime.h>

#include "gemm_common.h"

namespace dg {

// 1 / (1 + exp(-v)): exp overflows to infinity for large negative v and the
// reciprocal is then 0. Hardware exp2 and reciprocal, each within about an ulp.
__device__ __forceinline__ float sigmoid_f(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

// The tanh form of GELU, 0.5 z (1 + tanh(u)) with u = sqrt(2/pi) (z + 0.044715
// z^3), is z * sigmoid(2u).
constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kTanhB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_fn(float z) {
  if constexpr (ACT == 1) return fmaxf(z, 0.0f);
  if constexpr (ACT == 2) return 0.5f * z * (1.0f + erf_as7126(z * 0.70710678118654752f));
  if constexpr (ACT == 3) return z * sigmoid_f(z);
  if constexpr (ACT == 4) return z * sigmoid_f(kTanhA * z * __builtin_fmaf(kTanhB * z, z, 1.0f));
  return z;
}

// d act / dz. ReLU has 0 at 0.
//
// GELU: Phi(z) + z phi(z), which is 1 minus its value at -z; with a = |z| and
// e = exp(-a^2/2) the value at -a is e * (P(t)/2 - a / sqrt(2 pi)), where
// P(t) e is erfc(a / sqrt 2) by Abramowitz and Stegun 7.1.26 (the polynomial of
// erf_as7126), t = 1 / (1 + 0.3275911 a / sqrt 2): one exponential serves both
// terms, and both tails go to exactly 0 and 1. Absolute error: the polynomial's
// 7e-8, and up to 2.2e-7 from the roundings of t and of its alternating terms near
// t = 1 (2.9e-7 together at |z| = 0.067 with an exact reciprocal and exp2; 2.3e-7
// measured over every BF16 z).
//
// SiLU and the tanh form are z p(v), p = sigmoid(v), with v = z and v = 2u;
// their derivative p + z p (1 - p) v' is 1 minus its value at -z too. With
// a = |z|, e = exp(-v(a)) and t = 1 / (1 + e) the value at -a is
// e t (1 - a v'(a) t), which has no cancellation of 1 - p (there an absolute
// error of half an FP32 step of 1 would be multiplied by a v', up to 4e-7). In
// the tanh form both tails are exact from a = 30, where a is clamped before
// its powers can overflow.
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == 1) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == 2) {
    const float a = fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f * 0.70710678118654752f, a, 1.0f));
    float q = __builtin_fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
    q = __builtin_fmaf(q, t, 0.5f * 1.421413741f);
    q = __builtin_fmaf(q, t, 0.5f * -0.284496736f);
    q = __builtin_fmaf(q, t, 0.5f * 0.254829592f);
    const float e = __builtin_amdgcn_exp2f(-0.5f * 1.4426950408889634f * a * a);
    const float tail = e * __builtin_fmaf(q, t, -0.3989422804014327f * a);
    return z < 0.0f ? tail : 1.0f - tail;
  }
  if constexpr (ACT == 3 || ACT == 4) {
    float a = fabsf(z), v = a, adv = a;
    if constexpr (ACT == 4) {
      a = fminf(a, 30.0f);
      const float aa = a * a;
      v = kTanhA * a * __builtin_fmaf(kTanhB, aa, 1.0f);
      adv = kTanhA * a * __builtin_fmaf(3.0f * kTanhB, aa, 1.0f);
    }
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * v);
    const float t = __builtin_amdgcn_rcpf(1.0f + e);
    const float tail = e * t * __builtin_fmaf(-adv, t, 1.0f);
    return z < 0.0f ? tail : 1.0f - tail;
  }
  return 1.0f;
}

}  // namespace dg
