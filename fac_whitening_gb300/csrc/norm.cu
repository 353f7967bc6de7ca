// Layer norm forward and backward.
//
// Forward, one CTA per row: the mean, the sum of squared deviations, then y and (optionally) the
// 8-bit checkpoint of the normalised row, a warp per group of 128 columns.
// Backward: dx row by row (two sums over the row), and the sums over tokens of dy n and dy in
// slices of consecutive tokens, the slices added in order.
#include "act.cuh"
#include "kernels.cuh"

namespace gift {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float block_sum(float v, float *sh /* kNormThreads / 32 */) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) r += sh[i];
  return r;
}

template <int F, typename E>
__global__ void __launch_bounds__(kNormThreads) k_norm_forward(const E *__restrict__ x, int T, int d,
                                                               const float *__restrict__ gamma,
                                                               const float *__restrict__ beta, float eps,
                                                               E *__restrict__ y, float *__restrict__ mean_out,
                                                               float *__restrict__ rstd_out,
                                                               uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scales, int *status) {
  __shared__ float sh[kNormThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (d + kActGroup - 1) / kActGroup;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const E *xr = x + (size_t)t * d;
    float s = 0.0f;
    for (int c = threadIdx.x; c < d; c += kNormThreads) s += ld1(xr + c);
    const float mean = __fdiv_rn(block_sum(s, sh), (float)d);
    float q = 0.0f;
    for (int c = threadIdx.x; c < d; c += kNormThreads) {
      const float u = ld1(xr + c) - mean;
      q = fmaf(u, u, q);
    }
    const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(block_sum(q, sh), (float)d) + eps));
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[t] = mean;
      if (rstd_out) rstd_out[t] = rstd;
      if (!isfinite(mean) || !isfinite(rstd)) set_status(status, GIFT_ERR_NONFINITE);
    }
    for (int g = warp; g < groups; g += kNormThreads / 32) {
      float n[4];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = g * kActGroup + lane + 32 * i;
        n[i] = c < d ? (ld1(xr + c) - mean) * rstd : 0.0f;
        m = max(m, abs_bits(n[i]));
        if (c < d) st1(y + (size_t)t * d + c, fmaf(n[i], gamma ? gamma[c] : 1.0f, beta ? beta[c] : 0.0f));
      }
      if (codes) {
        const uint32_t sb = act_scale_byte<F>(warp_max_u32(m));
        const float inv = act_inv_scale(sb == kActBad ? 127u : sb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = g * kActGroup + lane + 32 * i;
          if (c < d) codes[(size_t)t * d + c] = pack1_fp8<F>(__fmul_rn(n[i], inv));
        }
        if (lane == 0) scales[(size_t)t * groups + g] = (uint8_t)sb;
      }
    }
  }
}

// The normalised element (t, c) from what the forward pass kept.
template <int F, typename E>
struct Saved {
  const E *x;             // or the checkpoint
  const uint8_t *codes, *scales;
  const float *mean, *rstd;
  int d, groups;
  __device__ __forceinline__ float at(int t, int c) const {
    const size_t i = (size_t)t * d + c;
    if (codes) return dec_fp8<F>(codes[i]) * act_scale(scales[(size_t)t * groups + c / kActGroup]);
    return (ld1(x + i) - mean[t]) * rstd[t];
  }
};

template <int F, typename E>
__global__ void __launch_bounds__(kNormThreads) k_norm_dx(const E *__restrict__ dy, const Saved<F, E> S, int T, int d,
                                                          const float *__restrict__ gamma, E *__restrict__ dx,
                                                          int *status) {
  __shared__ float sh[kNormThreads / 32];
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    float a = 0.0f, b = 0.0f;
    for (int c = threadIdx.x; c < d; c += kNormThreads) {
      const float h = ld1(dy + (size_t)t * d + c) * (gamma ? gamma[c] : 1.0f);
      a += h;
      b = fmaf(h, S.at(t, c), b);
    }
    a = __fdiv_rn(block_sum(a, sh), (float)d);
    b = __fdiv_rn(block_sum(b, sh), (float)d);
    const float rstd = S.rstd[t];
    if (threadIdx.x == 0 && !(isfinite(a) && isfinite(b) && isfinite(rstd))) set_status(status, GIFT_ERR_NONFINITE);
    for (int c = threadIdx.x; c < d; c += kNormThreads) {
      const float h = ld1(dy + (size_t)t * d + c) * (gamma ? gamma[c] : 1.0f);
      st1(dx + (size_t)t * d + c, rstd * (h - a - S.at(t, c) * b));
    }
  }
}

// partials of one slice of consecutive tokens: part[2 slice] = sum dy n, part[2 slice + 1] = sum dy
template <int F, typename E>
__global__ void __launch_bounds__(kNormThreads) k_norm_cols(const E *__restrict__ dy, const Saved<F, E> S, int T,
                                                            int d, int rows, float *__restrict__ part) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= d) return;
  const int t0 = blockIdx.y * rows, t1 = min(T, t0 + rows);
  float g = 0.0f, b = 0.0f;
  for (int t = t0; t < t1; ++t) {
    const float v = ld1(dy + (size_t)t * d + c);
    g = fmaf(v, S.at(t, c), g);
    b += v;
  }
  part[(size_t)(2 * blockIdx.y) * d + c] = g;
  part[(size_t)(2 * blockIdx.y + 1) * d + c] = b;
}

// sums over tokens of one matrix, in slices
template <typename E>
__global__ void __launch_bounds__(kNormThreads) k_col_sums(const E *__restrict__ x, int T, int d, int rows,
                                                           float *__restrict__ part) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= d) return;
  const int t0 = blockIdx.y * rows, t1 = min(T, t0 + rows);
  float s = 0.0f;
  for (int t = t0; t < t1; ++t) s += ld1(x + (size_t)t * d + c);
  part[(size_t)blockIdx.y * d + c] = s;
}

// out[c] = sum over slices of part[slice stride + c]
__global__ void __launch_bounds__(kNormThreads) k_sum_parts(const float *__restrict__ part, int slices, size_t stride,
                                                            int d, float *__restrict__ out) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= d) return;
  float s = 0.0f;
  for (int i = 0; i < slices; ++i) s += part[(size_t)i * stride + c];
  out[c] = s;
}

constexpr int kColRows = 128;   // tokens of a slice, at least

int col_rows(int T) {   // at most 256 slices
  const int r = (T + 255) / 256;
  return r < kColRows ? kColRows : r;
}

template <int F, typename E>
cudaError_t backward(const Launch &L, const NormBackward &a) {
  Saved<F, E> S;
  S.x = a.codes ? nullptr : static_cast<const E *>(a.x);
  S.codes = a.codes;
  S.scales = a.scales;
  S.mean = a.mean;
  S.rstd = a.rstd;
  S.d = a.d;
  S.groups = (a.d + kActGroup - 1) / kActGroup;
  const E *dy = static_cast<const E *>(a.dy);
  const int grid = a.T < L.sms * 8 ? a.T : L.sms * 8;
  k_norm_dx<F, E><<<grid, kNormThreads, 0, L.stream>>>(dy, S, a.T, a.d, a.gamma, static_cast<E *>(a.dx), L.status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dgamma && !a.dbeta)) return e;
  const int rows = col_rows(a.T), slices = (a.T + rows - 1) / rows, cb = (a.d + kNormThreads - 1) / kNormThreads;
  k_norm_cols<F, E><<<dim3(cb, slices), kNormThreads, 0, L.stream>>>(dy, S, a.T, a.d, rows, a.part);
  if (a.dgamma)
    k_sum_parts<<<cb, kNormThreads, 0, L.stream>>>(a.part, slices, (size_t)2 * a.d, a.d, a.dgamma);
  if (a.dbeta)
    k_sum_parts<<<cb, kNormThreads, 0, L.stream>>>(a.part + a.d, slices, (size_t)2 * a.d, a.d, a.dbeta);
  return cudaGetLastError();
}

template <int F, typename E>
cudaError_t forward(const Launch &L, const NormForward &a) {
  const int grid = a.T < L.sms * 8 ? a.T : L.sms * 8;
  k_norm_forward<F, E><<<grid, kNormThreads, 0, L.stream>>>(static_cast<const E *>(a.x), a.T, a.d, a.gamma, a.beta,
                                                            a.eps, static_cast<E *>(a.y), a.mean, a.rstd, a.codes,
                                                            a.scales, L.status);
  return cudaGetLastError();
}

}  // namespace

size_t norm_part_floats(int T, int d) {
  const int rows = col_rows(T);
  return (size_t)2 * ((T + rows - 1) / rows) * d;
}

size_t col_part_floats(int T, int d) { return norm_part_floats(T, d) / 2; }

cudaError_t launch_col_sums(const Launch &L, const void *x, bool bf16, int T, int d, float *part, float *out) {
  const int rows = col_rows(T), slices = (T + rows - 1) / rows, cb = (d + kNormThreads - 1) / kNormThreads;
  if (bf16)
    k_col_sums<<<dim3(cb, slices), kNormThreads, 0, L.stream>>>(static_cast<const __nv_bfloat16 *>(x), T, d, rows, part);
  else
    k_col_sums<<<dim3(cb, slices), kNormThreads, 0, L.stream>>>(static_cast<const float *>(x), T, d, rows, part);
  k_sum_parts<<<cb, kNormThreads, 0, L.stream>>>(part, slices, (size_t)d, d, out);
  return cudaGetLastError();
}

cudaError_t launch_norm_forward(const Launch &L, int fmt, bool bf16, const NormForward &a) {
  if (fmt == FMT_E4M3)
    return bf16 ? forward<FMT_E4M3, __nv_bfloat16>(L, a) : forward<FMT_E4M3, float>(L, a);
  return bf16 ? forward<FMT_E5M2, __nv_bfloat16>(L, a) : forward<FMT_E5M2, float>(L, a);
}

cudaError_t launch_norm_backward(const Launch &L, int fmt, bool bf16, const NormBackward &a) {
  if (fmt == FMT_E4M3)
    return bf16 ? backward<FMT_E4M3, __nv_bfloat16>(L, a) : backward<FMT_E4M3, float>(L, a);
  return bf16 ? backward<FMT_E5M2, __nv_bfloat16>(L, a) : backward<FMT_E5M2, float>(L, a);
}

}  // namespace gift
