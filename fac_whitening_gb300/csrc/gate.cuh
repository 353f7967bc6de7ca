// The gate's activation a(g) and its derivative.  With z = g (SiLU) or z = 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU's
// tanh form, 0.5 (1 + tanh(z / 2)) = 1 / (1 + exp(-z))) and s = 1 / (1 + exp(-z)):
//   a = g s,  a' = s + g z' s (1 - s);
// GELU: a = g Phi(g), a' = Phi(g) + g phi(g), Phi(g) = erfc(-g / sqrt 2) / 2 (no cancellation for negative g).
#pragma once

#include "common.cuh"

namespace gift {

enum GateFn { GATE_SILU = 0, GATE_GELU = 1, GATE_GELU_TANH = 2 };

// The hardware's exponential, of half the argument and squared: results below 2^-126 are denormal, where the instruction
// itself makes them 0 or takes twice as long.
__device__ __forceinline__ float exp_hw(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 0.72134752044448170f));
  return e * e;
}

// s, and 1 - s in `other`: with e = exp(-|z|), 1 / (1 + e) and e / (1 + e), so that the smaller one keeps what FP32 has below
// 2^-126 (g s is a normal number down to g = -91).  FP32 results take the library's expf and neither is a difference;
// those of BF16 calls the hardware's exponential, about 2^-20 off, 2^-12 of BF16's rounding.  Codes of h are made from those
// too: with expf as many of them change, within 1 %, and a call of 16384 x 1536 x 6144 takes 6 us more.  Both take the hardware's
// reciprocal, of 1 to 2, a unit in the last place off.  5003 x 1361 x 2731 BF16 backward 88.5 us with SiLU, 115 with GELU's
// tanh form; with s = 1 / (1 + exp(-z)), 0 from z = -87.3 on, 85 and 111.
template <bool ACCURATE>
__device__ __forceinline__ float sigmoid(float z, float &other) {
  const float e = ACCURATE ? expf(-fabsf(z)) : exp_hw(-fabsf(z));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  const float t = e * r, s = z >= 0.0f ? r : t;
  other = !ACCURATE ? 1.0f - s : z >= 0.0f ? t : r;
  return s;
}

constexpr float kTanhScale = 1.5957691216057308f;   // 2 sqrt(2 / pi)
__device__ __forceinline__ float tanh_inner(float g) { return kTanhScale * fmaf(0.044715f * g * g, g, g); }

template <int FN, bool ACCURATE>
__device__ __forceinline__ float gate_value(float g) {
  if (FN == GATE_GELU) return g * (0.5f * erfcf(g * -0.70710678118654752f));
  float other;
  return g * sigmoid<ACCURATE>(FN == GATE_SILU ? g : tanh_inner(g), other);
}

// a(g), and a'(g) in `slope`
template <int FN, bool ACCURATE>
__device__ __forceinline__ float gate_slope(float g, float &slope) {
  if (FN == GATE_GELU) {
    const float phi = 0.5f * erfcf(g * -0.70710678118654752f), e = -0.5f * g * g;
    slope = fmaf(g * 0.3989422804014327f, ACCURATE ? expf(e) : exp_hw(e), phi);
    return g * phi;
  }
  float other;
  const float s = sigmoid<ACCURATE>(FN == GATE_SILU ? g : tanh_inner(g), other), a = g * s;
  if (FN == GATE_SILU) {
    slope = fmaf(a, other, s);
  } else {   // z' may overflow where s is 0 or 1 already
    const float t = s * other;
    slope = t == 0.0f ? s : fmaf(g * (kTanhScale * fmaf(3.0f * 0.044715f * g, g, 1.0f)), t, s);
  }
  return a;
}

}  // namespace gift
