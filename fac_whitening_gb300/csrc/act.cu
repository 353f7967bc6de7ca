// The 8-bit activation checkpoint: encode and decode.
//
// One warp takes a group of 128 consecutive columns of one token: its amax, the scale exponent
// from the amax's bit pattern, the codes x 2^-k by the hardware's round-to-nearest-even,
// saturating conversion.  Both directions stream each byte once; HBM bounds them.
#include "act.cuh"
#include "kernels.cuh"

namespace gift {

namespace {

constexpr int kActThreads = 256;

template <int F, typename E>
__global__ void __launch_bounds__(kActThreads) k_act_encode(const E *__restrict__ x, int T, int d, int groups,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                            int *status) {
  const int lane = threadIdx.x & 31;
  const size_t warps = (size_t)gridDim.x * (kActThreads / 32), n = (size_t)T * groups;
  for (size_t w = (size_t)blockIdx.x * (kActThreads / 32) + (threadIdx.x >> 5); w < n; w += warps) {
    const size_t t = w / groups;
    const int c0 = (int)(w - t * groups) * kActGroup, len = min(kActGroup, d - c0);
    const size_t base = t * d + c0;
    float v[4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      v[i] = c < len ? ld1(x + base + c) : 0.0f;
      m = max(m, abs_bits(v[i]));
    }
    const uint32_t sb = act_scale_byte<F>(warp_max_u32(m));
    const float inv = act_inv_scale(sb == kActBad ? 127u : sb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      if (c < len) codes[base + c] = pack1_fp8<F>(__fmul_rn(v[i], inv));
    }
    if (lane == 0) {
      scales[w] = (uint8_t)sb;
      if (sb == kActBad) set_status(status, GIFT_ERR_NONFINITE);
    }
  }
}

template <int F, typename E>
__global__ void __launch_bounds__(kActThreads) k_act_decode(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, int T, int d,
                                                            int groups, E *__restrict__ out, int *status) {
  const int lane = threadIdx.x & 31;
  const size_t warps = (size_t)gridDim.x * (kActThreads / 32), n = (size_t)T * groups;
  for (size_t w = (size_t)blockIdx.x * (kActThreads / 32) + (threadIdx.x >> 5); w < n; w += warps) {
    const size_t t = w / groups;
    const int c0 = (int)(w - t * groups) * kActGroup, len = min(kActGroup, d - c0);
    const size_t base = t * d + c0;
    const uint32_t sb = scales[w];
    const float s = act_scale(sb);
    for (int c = lane; c < len; c += 32) st1(out + base + c, __fmul_rn(dec_fp8<F>(codes[base + c]), s));
    if (lane == 0 && sb == kActBad) set_status(status, GIFT_ERR_NONFINITE);
  }
}

int act_grid(const Launch &L, size_t groups) {
  const size_t ctas = (groups + kActThreads / 32 - 1) / (kActThreads / 32);
  return (int)(ctas < (size_t)L.sms * 8 ? ctas : (size_t)L.sms * 8);
}

template <int F, typename E>
cudaError_t encode(const Launch &L, const void *x, int T, int d, uint8_t *codes, uint8_t *scales) {
  const int groups = (d + kActGroup - 1) / kActGroup;
  k_act_encode<F, E><<<act_grid(L, (size_t)T * groups), kActThreads, 0, L.stream>>>(
      static_cast<const E *>(x), T, d, groups, codes, scales, L.status);
  return cudaGetLastError();
}

template <int F, typename E>
cudaError_t decode(const Launch &L, const uint8_t *codes, const uint8_t *scales, int T, int d, void *out) {
  const int groups = (d + kActGroup - 1) / kActGroup;
  k_act_decode<F, E><<<act_grid(L, (size_t)T * groups), kActThreads, 0, L.stream>>>(codes, scales, T, d, groups,
                                                                                    static_cast<E *>(out), L.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_act_encode(const Launch &L, int fmt, const void *x, bool bf16, int T, int d, uint8_t *codes,
                              uint8_t *scales) {
  if (fmt == FMT_E4M3)
    return bf16 ? encode<FMT_E4M3, __nv_bfloat16>(L, x, T, d, codes, scales)
                : encode<FMT_E4M3, float>(L, x, T, d, codes, scales);
  return bf16 ? encode<FMT_E5M2, __nv_bfloat16>(L, x, T, d, codes, scales)
              : encode<FMT_E5M2, float>(L, x, T, d, codes, scales);
}

cudaError_t launch_act_decode(const Launch &L, int fmt, const uint8_t *codes, const uint8_t *scales, int T, int d,
                              void *out, bool bf16) {
  if (fmt == FMT_E4M3)
    return bf16 ? decode<FMT_E4M3, __nv_bfloat16>(L, codes, scales, T, d, out)
                : decode<FMT_E4M3, float>(L, codes, scales, T, d, out);
  return bf16 ? decode<FMT_E5M2, __nv_bfloat16>(L, codes, scales, T, d, out)
              : decode<FMT_E5M2, float>(L, codes, scales, T, d, out);
}

}  // namespace gift
