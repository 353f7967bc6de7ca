// Weight gradient from an 8-bit checkpoint, dW = delta^T v: FP32 SIMT.
//
// 64 x 64 tiles of dW, 16 tokens per step through shared memory, 4 x 4 outputs per thread; the
// running sums are folded into the totals every 256 tokens, so that rounding grows with the
// number of folds and not with T.
#include "act.cuh"
#include "kernels.cuh"

namespace gift {

namespace {

constexpr int kWTile = 64, kWStep = 16, kWThreads = 256, kWFold = 256;

template <int F, typename E>
__global__ void __launch_bounds__(kWThreads) k_weight_grad_simt(const E *__restrict__ delta,
                                                                const uint8_t *__restrict__ codes,
                                                                const uint8_t *__restrict__ scales, int T, int d_out,
                                                                int d_in, const float *__restrict__ gamma,
                                                                const float *__restrict__ beta,
                                                                const float *__restrict__ db, float *__restrict__ dW) {
  __shared__ float sa[kWStep][kWTile], sb[kWStep][kWTile];
  const int i0 = blockIdx.x * kWTile, o0 = blockIdx.y * kWTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int groups = (d_in + kActGroup - 1) / kActGroup;
  float acc[4][4] = {}, tot[4][4] = {};
  for (int t0 = 0; t0 < T; t0 += kWStep) {
#pragma unroll
    for (int j = 0; j < kWStep * kWTile / kWThreads; ++j) {
      const int q = threadIdx.x + j * kWThreads, r = q / kWTile, c = q % kWTile, t = t0 + r;
      sa[r][c] = (t < T && o0 + c < d_out) ? ld1(delta + (size_t)t * d_out + o0 + c) : 0.0f;
      sb[r][c] = (t < T && i0 + c < d_in)
                     ? dec_fp8<F>(codes[(size_t)t * d_in + i0 + c]) *
                           act_scale(scales[(size_t)t * groups + (i0 + c) / kActGroup])
                     : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kWStep; ++r)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(sa[r][ty + 16 * u], sb[r][tx + 16 * v], acc[u][v]);
    __syncthreads();
    if ((t0 + kWStep) % kWFold == 0 || t0 + kWStep >= T) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          tot[u][v] += acc[u][v];
          acc[u][v] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int o = o0 + ty + 16 * u;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = i0 + tx + 16 * v;
      if (o >= d_out || i >= d_in) continue;
      float w = gamma ? tot[u][v] * gamma[i] : tot[u][v];
      if (beta) w = fmaf(beta[i], db[o], w);
      dW[(size_t)o * d_in + i] = w;
    }
  }
}

template <int F, typename E>
cudaError_t simt(const Launch &L, const WeightGrad &a, const float *db) {
  const dim3 grid((a.d_in + kWTile - 1) / kWTile, (a.d_out + kWTile - 1) / kWTile);
  k_weight_grad_simt<F, E><<<grid, kWThreads, 0, L.stream>>>(static_cast<const E *>(a.delta), a.codes, a.scales, a.T,
                                                             a.d_out, a.d_in, a.gamma, a.beta, db, a.dW);
  return cudaGetLastError();
}

}  // namespace

WeightGradWs weight_grad_layout(const Launch &L, bool bf16, int T, int d_out, int d_in) {
  (void)L; (void)bf16; (void)d_in;
  WeightGradWs w;
  w.part_floats = col_part_floats(T, d_out);
  return w;
}

cudaError_t launch_weight_grad(const Launch &L, int fmt, bool bf16, const WeightGrad &a) {
  const float *db = nullptr;
  if (a.db || a.beta) {
    float *out = a.db ? a.db : a.db_ws;
    const cudaError_t e = launch_col_sums(L, a.delta, bf16, a.T, a.d_out, a.part, out);
    if (e != cudaSuccess) return e;
    db = out;
  }
  if (fmt == FMT_E4M3) return bf16 ? simt<FMT_E4M3, __nv_bfloat16>(L, a, db) : simt<FMT_E4M3, float>(L, a, db);
  return bf16 ? simt<FMT_E5M2, __nv_bfloat16>(L, a, db) : simt<FMT_E5M2, float>(L, a, db);
}

}  // namespace gift
