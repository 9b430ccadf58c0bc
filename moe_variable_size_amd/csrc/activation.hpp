// The dense layers' activations and their derivatives.
#pragma once
#include <type_traits>

#include "common.hpp"

namespace moe {

MOE_DEV float sigmoidf(float t) { return __builtin_amdgcn_rcpf(1.f + __expf(-t)); }
constexpr float kTanhC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// The normal distribution's upper tail Q(x) = 1 - Phi(x) at x = |z|, and e = exp(-x^2 / 2); z Phi(z) =
// max(z, 0) - x Q(x).  Q = e G with G(x) = erfcx(x / sqrt 2) / 2, fitted as a polynomial in t = 1 / (1 + 0.3 x)
// by least squares of the relative error on Chebyshev nodes over 0 <= x <= 14 (beyond, e is 0; the fit
// alone is off by 7e-8).  1 + erf(z / sqrt 2) would cancel to nothing in the tail; here what grows is the
// exponent's rounding, three times 2^-24 x^2 / 2: relative error of Q at most (1.5 x^2 + 17) 2^-24, 4e-7
// found below x = 1, 2e-6 up to 6, 8e-6 up to 13.  One exponential, one reciprocal, 8 multiply-adds.
MOE_DEV float normal_tail(float z, float &e) {
  const float x = fabsf(z), t = __builtin_amdgcn_rcpf(fmaf(0.3f, x, 1.f));
  e = __builtin_amdgcn_exp2f(-0.72134752f * x * x);  // 1 / (2 ln 2)
  float g = 3.88709204e-2f;
  g = fmaf(g, t, -1.71443555e-1f);
  g = fmaf(g, t, 2.33107471e-1f);
  g = fmaf(g, t, -8.12823041e-2f);
  g = fmaf(g, t, 1.45609827e-1f);
  g = fmaf(g, t, 9.34725846e-2f);
  g = fmaf(g, t, 1.22204592e-1f);
  g = fmaf(g, t, 1.19451402e-1f);
  g = fmaf(g, t, 9.09630867e-6f);
  return e * g;
}

template <int ACT>
MOE_DEV float act_fwd(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    const float q = normal_tail(z, e);
    // above 14.5 x Q is far below half a step of z; and inf * 0 would make gelu(inf) a NaN
    return z > 14.5f ? z : fmaf(-fabsf(z), q, fmaxf(z, 0.f));
  }
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == MOE_ACT_GELU_TANH)
    return z * sigmoidf(2.f * kTanhC * (z + kTanhA * z * z * z));
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoidf(z);
  return z;
}

template <int ACT>
MOE_DEV float act_grad(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    const float q = normal_tail(z, e);
    return fmaf(z * 0.3989422804f, e, z < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    const float s = sigmoidf(2.f * kTanhC * (z + kTanhA * z * z * z)), t = s * (1.f - s);
    // far out t is 0 and its factor may overflow
    return t == 0.f ? s : s + z * t * (2.f * kTanhC * (1.f + 3.f * kTanhA * z * z));
  }
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoidf(z);
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

// act(z) of an activation known at run time
MOE_DEV float act_fwd_of(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return act_fwd<MOE_ACT_RELU>(z);
    case MOE_ACT_GELU: return act_fwd<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_fwd<MOE_ACT_GELU_TANH>(z);
    case MOE_ACT_SILU: return act_fwd<MOE_ACT_SILU>(z);
    default: return z;
  }
}

// f(integral_constant<act>)
template <class F>
void by_act(int act, F &&f) {
  switch (act) {
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>()); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>()); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>()); break;
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>()); break;
    default: f(std::integral_constant<int, MOE_ACT_NONE>());
  }
}

}  // namespace moe
