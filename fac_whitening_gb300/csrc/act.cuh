// Device helpers of the 8-bit activation checkpoint, shared by its encode and decode, the layer
// norm and the weight gradient.
#pragma once

#include "common.cuh"

namespace gift {

constexpr int kActGroup = 128;   // columns of a token that share a scale
constexpr int kActKMin = -110;   // smallest scale exponent: every value stays a normal FP32 or an exact BF16 one
constexpr uint32_t kActBad = 255u;   // scale byte of a group that holds NaN or Inf

template <int F>
__host__ __device__ constexpr int act_emax() { return F == FMT_E4M3 ? 8 : 15; }   // exponent of FMAX

// Scale byte of a group from the bit pattern of its amax.  FMAX = 1.75 2^EMAX, so amax <= FMAX 2^k
// first holds at k = E - EMAX, E the exponent of amax, or one above when its significand is over
// 1.75: integer arithmetic, no rounding.
template <int F>
__device__ __forceinline__ uint32_t act_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kActBad;
  int k = (int)(amax_bits >> 23) - 127 - act_emax<F>() + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  k = min(max(k, kActKMin), 127 - act_emax<F>());
  return (uint32_t)(k + 127);
}
// 2^-k, what an element is multiplied with before it is rounded (k in [-110, 119]: normal)
__device__ __forceinline__ float act_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^k; NaN for a marked group
__device__ __forceinline__ float act_scale(uint32_t byte) {
  return byte == kActBad ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float ld1(const float *p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float *p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace gift
