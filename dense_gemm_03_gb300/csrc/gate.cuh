// gate.cuh -- the activations of a gated block, f(g) and f'(g) in fp32.
//
//   silu       f = g s,             s = 1 / (1 + e^-g);      f' = s (1 + g (1 - s))
//   gelu       f = g P,             P = 1 - Q(g), P = Q(-g) for g < 0;   f' = P + g phi(g)
//              Q(g) = erfc(|g| / sqrt 2) / 2 = e^(-g^2/2) t p(t) / 2,  t = 1 / (1 + 0.44 |g| / sqrt 2),
//              p of degree 7 fitted (least largest relative error, 1.8e-7) to the scaled
//              function e^(x^2) erfc(x) over 0 <= x <= 10, past which e^(-x^2) is zero.
//              With erfcf instead the epilogue of a 256 x 128 tile took 4.8 us, not 1.7
//   gelu_tanh  f = g s,             s = 1 / (1 + e^-2z) = (1 + tanh z) / 2,
//              z = sqrt(2/pi) (g + 0.044715 g^3);           f' = s + 2 g z' s (1 - s)
//   relu       f = max(g, 0);                                f' = 1 for g > 0, else 0
// f is exact in the tails (no difference of near-equal numbers): a large negative g
// makes e^-g infinite and s zero.  In f' 1 - s is off by 2^-25 where s is near 1, times |g| < 17 (it
// is zero past that) beside an f' of about 1.  A NaN stays a NaN.  Results below 2^-126 may be
// zero on the way: s, e^-x and 1 / x are one instruction each then.
#pragma once
#include <type_traits>

#include "gemm.h"

namespace gb300 {

// e^-x = 2^(-x / ln 2) and 1 / x, with relative errors of about 2^-22 (1 + |x| / 4) and 2^-23.
__device__ __forceinline__ float gate_exp_neg(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float gate_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// s = 1 / (1 + e^-x); 0 where e^-x passes 2^126.
__device__ __forceinline__ float gate_logistic(float x) {
  return gate_inverse(1.0f + gate_exp_neg(x));
}

constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// f(g), and f'(g) into d.
template <int ACT>
__device__ __forceinline__ float gate_both(float g, float& d) {
  if (ACT == GEMM_ACT_SILU) {
    const float s = gate_logistic(g);
    d = s * fmaf(g, 1.0f - s, 1.0f);
    return g * s;
  }
  if (ACT == GEMM_ACT_GELU) {
    const float x = 0.7071067811865476f * fabsf(g);
    const float e = gate_exp_neg(x * x), t = gate_inverse(fmaf(0.44f, x, 1.0f));
    float q = 0.07122123653597495f;
    q = fmaf(q, t, -0.2779385877587885f);
    q = fmaf(q, t, 0.2966708364139223f);
    q = fmaf(q, t, -0.02016481289303846f);
    q = fmaf(q, t, 0.21580346214090299f);
    q = fmaf(q, t, 0.21731635716162814f);
    q = fmaf(q, t, 0.2488707024307475f);
    q = fmaf(q, t, 0.2482209868978177f);
    q *= 0.5f * t * e;
    const float P = g < 0.0f ? q : 1.0f - q;
    d = fmaf(g, 0.3989422804014327f * e, P);
    return g * P;
  }
  if (ACT == GEMM_ACT_GELU_TANH) {
    const float g2 = g * g;
    const float s = gate_logistic(2.0f * kGeluC * g * fmaf(kGeluA, g2, 1.0f));
    const float dz = 2.0f * kGeluC * fmaf(3.0f * kGeluA, g2, 1.0f);
    // past any use of the product dz could overflow: s or 1 - s is zero there
    d = fabsf(g) > 16.0f ? s : fmaf(g * dz, s * (1.0f - s), s);
    return g * s;
  }
  d = g > 0.0f || g != g ? 1.0f : 0.0f;
  return g > 0.0f || g != g ? g : 0.0f;
}

template <int ACT>
__device__ __forceinline__ float gate_value(float g) {
  float d;
  return gate_both<ACT>(g, d);
}

// fn(constant) with the constant the activation `act` is.
template <class F>
__device__ __forceinline__ void gate_dispatch(int act, F&& fn) {
  switch (act) {
    case GEMM_ACT_SILU: fn(std::integral_constant<int, GEMM_ACT_SILU>{}); break;
    case GEMM_ACT_GELU: fn(std::integral_constant<int, GEMM_ACT_GELU>{}); break;
    case GEMM_ACT_GELU_TANH: fn(std::integral_constant<int, GEMM_ACT_GELU_TANH>{}); break;
    default: fn(std::integral_constant<int, GEMM_ACT_RELU>{}); break;
  }
}

}  // namespace gb300
