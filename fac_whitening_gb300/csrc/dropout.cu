// Dropout by itself: y = residual + drop(x + bias), and its backward pass dx = drop(dy), dbias = sum_t dx.
//
// HBM bounds it.  A warp keeps one piece of 256 columns (8 a lane: one counter) and walks down the rows of its CTA's
// slice, two at a time so that their loads are in flight together; the bits are drawn where they are used.  32768 x 4096
// BF16 130 us forward with bias and residual (6.2 TB/s), 105 backward with dbias (5.1); 16384 x 1536 31 and 29.  With pieces
// of 512 columns, 16 a lane, 173 and 122: half the warps fit.
#include "act.cuh"
#include "dropout.cuh"
#include "kernels.cuh"

namespace gift {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kC = 8, kCols = 32 * kC;   // columns of a lane, of a piece
constexpr int kRows = 2;                 // rows of a step of a warp

// Drop a lane's values of a row: VEC, its own columns; otherwise value e is column 32 e + lane, whose bit lane
// (32 e + lane) / 8 drew.
template <bool VEC>
__device__ __forceinline__ void drop(const Draw &d, float2 *v, uint32_t row, uint32_t c0, int lane) {
  if (VEC) {
    d.apply8(v, row, c0 / 8 + lane);
    return;
  }
  const uint32_t m = d.keep8(row, c0 / 8 + lane);
#pragma unroll
  for (int k = 0; k < kC / 2; ++k) {
    const uint32_t a = __shfl_sync(0xFFFFFFFFu, m, 8 * k + (lane >> 3));
    const uint32_t b = __shfl_sync(0xFFFFFFFFu, m, 8 * k + 4 + (lane >> 3));
    v[k].x = a >> (lane & 7) & 1u ? v[k].x * d.scale : 0.0f;
    v[k].y = b >> (lane & 7) & 1u ? v[k].y * d.scale : 0.0f;
  }
}

struct Args {
  const void *x, *residual;   // residual nullable
  const float *bias;          // nullable
  void *y;
  int T, d, rows;             // rows of a slice
  Dropout drop;
  float *part;                // nullable: [slices][d] sums of y over the slice's rows
};

template <typename E, bool VEC, bool SUMS>
__global__ void __launch_bounds__(kThreads) k_dropout(const Args a) {
  __shared__ float sh[SUMS ? kWarps : 1][SUMS ? kC * 33 : 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kCols, n = a.d - c0;
  const int t0 = blockIdx.y * a.rows, t1 = min(a.T, t0 + a.rows);
  const Draw draw(a.drop);
  float2 bias[kC / 2], sum[kC / 2];
#pragma unroll
  for (int k = 0; k < kC / 2; ++k) {
    bias[k] = sum[k] = both(0.0f);
    if (!SUMS && a.bias) {
      const int c = piece_col<VEC, kC>(lane, 2 * k), c1 = piece_col<VEC, kC>(lane, 2 * k + 1);
      bias[k] = make_float2(c < n ? a.bias[c0 + c] : 0.0f, c1 < n ? a.bias[c0 + c1] : 0.0f);
    }
  }
  const E *x = static_cast<const E *>(a.x) + c0, *res = static_cast<const E *>(a.residual);
  for (int t = t0 + w; t < t1; t += kRows * kWarps) {
    Raw<E, kC> r[kRows], q[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const size_t at = (size_t)(t + u * kWarps) * a.d;
      if (t + u * kWarps >= t1) break;
      load_piece<VEC>(x + at, n, lane, r[u]);
      if (!SUMS && res) load_piece<VEC>(res + c0 + at, n, lane, q[u]);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int row = t + u * kWarps;
      if (row >= t1) break;
      float2 v[kC / 2];
#pragma unroll
      for (int k = 0; k < kC / 2; ++k) v[k] = SUMS ? r[u].pair(k) : add2(r[u].pair(k), bias[k]);
      if (draw.below) drop<VEC>(draw, v, row, c0, lane);
#pragma unroll
      for (int k = 0; k < kC / 2; ++k) {
        if (SUMS) sum[k] = add2(sum[k], v[k]);
        else if (res) v[k] = add2(v[k], q[u].pair(k));
      }
      store_piece<VEC, kC>(static_cast<E *>(a.y) + c0 + (size_t)row * a.d, n, lane, v);
    }
  }
  if constexpr (SUMS) {
    if (!a.part) return;
#pragma unroll
    for (int e = 0; e < kC; ++e) sh[w][33 * e + lane] = e & 1 ? sum[e / 2].y : sum[e / 2].x;
    __syncthreads();
    for (int c = threadIdx.x; c < kCols && c < n; c += kThreads) {
      const int at = VEC ? 33 * (c % kC) + c / kC : 33 * (c / 32) + c % 32;
      float v = sh[0][at];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) v += sh[k][at];
      a.part[(size_t)blockIdx.y * a.d + c0 + c] = v;
    }
  }
}

// Slices of rows: about eight CTAs per SM with all pieces, a step of the CTA's warps at least.
int slices_of(int sms, int T, int d) {
  const int pieces = (d + kCols - 1) / kCols, most = (T + kRows * kWarps - 1) / (kRows * kWarps);
  const int s = (8 * sms + pieces - 1) / pieces;
  return s < most ? s : most;
}

template <typename E, bool SUMS>
cudaError_t launch(const Launch &L, const Args &a, int slices) {
  const dim3 grid((a.d + kCols - 1) / kCols, slices);
  const bool vec = rows_vec(a.d, a.x, nullptr) && rows_vec(a.d, a.y, nullptr) && rows_vec(a.d, a.residual, nullptr);
  if (vec) k_dropout<E, true, SUMS><<<grid, kThreads, 0, L.stream>>>(a);
  else k_dropout<E, false, SUMS><<<grid, kThreads, 0, L.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t dropout_part_floats(int sms, int T, int d) { return (size_t)slices_of(sms, T, d) * d; }

cudaError_t launch_dropout_forward(const Launch &L, bool bf16, const DropoutCall &c) {
  Args a{};
  a.x = c.x;
  a.residual = c.residual;
  a.bias = c.bias;
  a.y = c.y;
  a.T = c.T;
  a.d = c.d;
  a.drop = Dropout{c.rng, c.below, c.site, 65536.0f / (float)(65536 - c.below)};
  const int s = slices_of(L.sms, c.T, c.d);
  a.rows = (c.T + s - 1) / s;
  return bf16 ? launch<__nv_bfloat16, false>(L, a, s) : launch<float, false>(L, a, s);
}

cudaError_t launch_dropout_backward(const Launch &L, bool bf16, const DropoutCall &c) {
  Args a{};
  a.x = c.x;
  a.y = c.y;
  a.T = c.T;
  a.d = c.d;
  a.drop = Dropout{c.rng, c.below, c.site, 65536.0f / (float)(65536 - c.below)};
  a.part = c.dbias ? c.part : nullptr;
  const int s = slices_of(L.sms, c.T, c.d);
  a.rows = (c.T + s - 1) / s;
  const cudaError_t e = bf16 ? launch<__nv_bfloat16, true>(L, a, s) : launch<float, true>(L, a, s);
  if (e != cudaSuccess || !c.dbias) return e;
  return launch_sum_parts(L, c.part, s, c.d, c.dbias);
}

}  // namespace gift
