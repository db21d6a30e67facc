// glu_act.cuh -- the activations of the gated feed-forward block and their derivatives.
//
// Exponential and reciprocal are the hardware's (ex2.approx, rcp.approx: 2^-22 and 2^-23 of their values). What they
// give is rounded to BF16 (2^-9) right after, directly or as H, dg and du.
#pragma once

#include "common.cuh"
#include "gemm.h"

namespace dtcp {

__device__ __forceinline__ float nan_max0(float v) {  // max(v, 0), NaN for NaN
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(0.0f));
  return r;
}

// act(g). SiLU: g / (1 + exp(-g)); GELU, tanh form, as g / (1 + exp(-2 v)), v = sqrt(2/pi) (g + 0.044715 g^3).
// An exponential that overflows gives 1 / inf = 0.
__device__ __forceinline__ float glu_act(float g, int act) {
  if (act == GEMM_GLU_SILU) return g * rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * g));
  if (act == GEMM_GLU_GELU_TANH) {
    const float t = fmaf(0.044715f * g, g * g, g);
    return g * rcp_approx(1.0f + ex2_approx(-2.302208198144325f * t));
  }
  return nan_max0(g);
}

// act(g) and act'(g).
__device__ __forceinline__ void glu_act_grad(float g, int act, float& a, float& da) {
  if (act == GEMM_GLU_SILU) {
    const float s = rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * g));
    a = g * s;
    da = s * fmaf(g, 1.0f - s, 1.0f);
  } else if (act == GEMM_GLU_GELU_TANH) {
    const float t = fmaf(0.044715f * g, g * g, g);
    const float s = rcp_approx(1.0f + ex2_approx(-2.302208198144325f * t));
    a = g * s;
    const float slope = s * (1.0f - s);  // 0 once s is 0 or 1, whatever the polynomial's size
    const float dv = 1.5957691216057308f * fmaf(0.134145f * g, g, 1.0f);
    da = slope == 0.0f ? s : fmaf(g * slope, dv, s);
  } else {
    a = nan_max0(g);
    da = g > 0.0f ? 1.0f : (g != g ? g : 0.0f);
  }
}

}  // namespace dtcp
