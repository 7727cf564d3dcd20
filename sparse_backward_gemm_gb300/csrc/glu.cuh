// The gated feed-forward block's activations, in f32 (sm_103a).
#pragma once

#include "common.cuh"

namespace collider {

constexpr int kGluSilu = 0, kGluGeluTanh = 1;

// SiLU: a(g) = g p, p = sigmoid(g), a' = p (1 + g (1 - p)).
// GELU (tanh form): with z = c (g + k g^3), (1 + tanh z) / 2 = sigmoid(2 z) = p,
// so a(g) = g p and a' = p + 2 g p (1 - p) c (1 + 3 k g^2): one exponential and
// one reciprocal either way, and no cancellation for g far below 0.
// The exponential and the reciprocal are the hardware's (about 2^-22 of the
// value each): every result is rounded to bf16.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int ACT>
__device__ __forceinline__ float glu_gate(float g) {
  constexpr float log2e = 1.4426950408889634f, c2 = 2.f * 0.7978845608028654f, k = 0.044715f;
  const float z = ACT == kGluSilu ? -log2e * g : (-log2e * c2) * g * fmaf(k * g, g, 1.f);
  return rcp_approx(1.f + ex2_approx(z));
}
template <int ACT>
__device__ __forceinline__ float glu_act(float g) {
  return g * glu_gate<ACT>(g);
}
// a(g) and a'(g)
template <int ACT>
__device__ __forceinline__ void glu_both(float g, float* a, float* da) {
  const float p = glu_gate<ACT>(g);
  *a = g * p;
  if (ACT == kGluSilu) {
    *da = p * fmaf(g, 1.f - p, 1.f);
  } else {
    constexpr float c2 = 2.f * 0.7978845608028654f, k3 = 3.f * 0.044715f;
    // (|g| up to 64: from 20 on p is 0 or 1 and the term 0, and its square must not become an infinity)
    const float h = fminf(fabsf(g), 64.f);
    *da = fmaf(*a * (1.f - p), c2 * fmaf(k3 * h, h, 1.f), p);
  }
}

}  // namespace collider
