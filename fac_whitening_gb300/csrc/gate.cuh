// The gate's activation a(g) and its derivative.  With z = g (SiLU) or z = 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's
// tanh form, 0.5 (1 + tanh(z / 2)) = 1 / (1 + exp(-z))) and s = 1 / (1 + exp(-z)):
//   a = g s,  a' = s + g z' s (1 - s);
// GELU: a = g Phi(g), a' = Phi(g) + g phi(g), Phi(g) = erfc(-g / sqrt 2) / 2 (no cancellation for negative g).
#pragma once

#include "common.cuh"

namespace gift {

enum GateFn { GATE_SILU = 0, GATE_GELU = 1, GATE_GELU_TANH = 2 };

// FP32 results take the library's expf and division (a few units in the last place); results that are rounded to
// BF16 the hardware's exponential and reciprocal (about 2^-21 off, 2^-13 of BF16's rounding).
template <bool ACCURATE>
__device__ __forceinline__ float sigmoid(float z) {
  if (ACCURATE) return 1.0f / (1.0f + expf(-z));
  return __fdividef(1.0f, 1.0f + __expf(-z));   // 0 where the exponential is infinite or past 2^126
}

template <int FN, bool ACCURATE>
__device__ __forceinline__ float gate_value(float g) {
  if (FN == GATE_GELU) return g * (0.5f * erfcf(g * -0.70710678118654752f));
  const float c = 1.5957691216057308f;
  return g * sigmoid<ACCURATE>(FN == GATE_SILU ? g : c * fmaf(0.044715f * g * g, g, g));
}

// a(g), and a'(g) in `slope`
template <int FN, bool ACCURATE>
__device__ __forceinline__ float gate_slope(float g, float &slope) {
  if (FN == GATE_GELU) {
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f), e = -0.5f * g * g;
    slope = fmaf(g * 0.3989422804014327f, ACCURATE ? expf(e) : __expf(e), phi);
    return g * phi;
  }
  const float c = 1.5957691216057308f;
  const float s = sigmoid<ACCURATE>(FN == GATE_SILU ? g : c * fmaf(0.044715f * g * g, g, g));
  const float t = s * (1.0f - s);
  // z' may overflow where s is 0 or 1 already
  if (FN == GATE_SILU) slope = fmaf(g, t, s);
  else slope = t == 0.0f ? s : fmaf(g * (c * fmaf(3.0f * 0.044715f * g, g, 1.0f)), t, s);
  return g * s;
}

}  // namespace gift
