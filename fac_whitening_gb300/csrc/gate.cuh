// The gate's activation a(g) and its derivative.  With z = g (SiLU) or z = 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's
// tanh form, 0.5 (1 + tanh(z / 2)) = 1 / (1 + exp(-z))) and s = 1 / (1 + exp(-z)):
//   a = g s,  a' = s + g z' s (1 - s);
// GELU: a = g Phi(g), a' = Phi(g) + g phi(g), Phi(g) = erfc(-g / sqrt 2) / 2 (no cancellation for negative g).
#pragma once

#include "common.cuh"

namespace gift {

enum GateFn { GATE_SILU = 0, GATE_GELU = 1, GATE_GELU_TANH = 2 };

// FP32 results take the library's expf; results that are rounded to BF16 the hardware's exponential (about 2^-21 off,
// 2^-13 of BF16's rounding; results below 2^-126 are 0, where s is 1 to the last place).  Both take the hardware's
// reciprocal, a unit in the last place off.
template <bool ACCURATE>
__device__ __forceinline__ float sigmoid(float z) {
  float e, s;
  if (ACCURATE) e = expf(-z);
  else asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));   // 0 where e is infinite
  return s;
}

constexpr float kTanhScale = 1.5957691216057308f;   // 2 sqrt(2 / pi)
__device__ __forceinline__ float tanh_inner(float g) { return kTanhScale * fmaf(0.044715f * g * g, g, g); }

template <int FN, bool ACCURATE>
__device__ __forceinline__ float gate_value(float g) {
  if (FN == GATE_GELU) return g * (0.5f * erfcf(g * -0.70710678118654752f));
  return g * sigmoid<ACCURATE>(FN == GATE_SILU ? g : tanh_inner(g));
}

// a(g), and a'(g) in `slope`
template <int FN, bool ACCURATE>
__device__ __forceinline__ float gate_slope(float g, float &slope) {
  if (FN == GATE_GELU) {
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f), e = -0.5f * g * g;
    slope = fmaf(g * 0.3989422804014327f, ACCURATE ? expf(e) : __expf(e), phi);
    return g * phi;
  }
  const float s = sigmoid<ACCURATE>(FN == GATE_SILU ? g : tanh_inner(g)), a = g * s;
  if (FN == GATE_SILU) {
    slope = fmaf(a, 1.0f - s, s);
  } else {   // z' may overflow where s is 0 or 1 already
    const float t = s * (1.0f - s);
    slope = t == 0.0f ? s : fmaf(g * (kTanhScale * fmaf(3.0f * 0.044715f * g, g, 1.0f)), t, s);
  }
  return a;
}

}  // namespace gift
