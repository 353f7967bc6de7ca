// Layer norm forward and backward.
//
// Both hold a row's share in registers (pieces of act.cuh) and move each byte once: forward 4 bytes an
// element for BF16, 5 with the checkpoint; backward 6, or 5 from the checkpoint.  A row belongs to a
// group of warps (row_plan, forward_plan, backward_plan), and the next row is loaded before this one's
// sums are waited for.
//
// Forward: the mean and the squared deviations from it, reduced from registers; y and the checkpoint are
// written from them.  32768 x 4096 BF16: 91 us, 5.9 TB/s; with the checkpoint 111 us, 6.0 TB/s: HBM, at
// 0.87 of the copy rate; 16384 x 1536 with the checkpoint 26.8 us, 4.7 TB/s; 16384 x 4096 FP32 97 us, 5.5
// TB/s, with the checkpoint 108 us, 5.6 TB/s.  Element accesses: 4099 x 7001 BF16 72 us, 1.6 TB/s.
//
// Backward: sums over a row (h and h n) for dx, and sums over tokens (dy n and dy) for the gain's and
// offset's gradients.  The latter stay in the registers of the thread that owns the column: a CTA
// takes every gridDim-th row, adds its row groups' sums through shared memory at the end and writes
// one partial; k_norm_sums adds the partials.  The order is fixed by the shape, the accesses (rows_vec)
// and the grid.  32768 x 4096 BF16: 171 us, 4.7 TB/s (dx alone, same kernel: 158); 16384 x 1536 from
// the checkpoint 34 us, 3.7 TB/s.  One row ahead in registers, 12 to 16 warps per SM up to 4096 columns:
// at most 32 KB in flight, which wait at each row's barrier; a third of the issue slots are used.  From
// 4097 columns a CTA is one row and the registers hold one CTA per SM, 9 to 16 warps: 32768 x 4608 BF16
// 261 us (3.5 TB/s), 5120 273, 6144 297, 16384 x 8192 181 (4.5 TB/s).  Rings of per-thread asynchronous
// copies in shared memory and batches of two to four rows per reduction were measured and were no faster.
#include "act.cuh"
#include "kernels.cuh"

namespace gift {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Two sums over the warp in six shuffles: the halves of the warp take one each after the first step.
__device__ __forceinline__ float2 warp_sum2(float2 v) {
  const bool upper = threadIdx.x & 16;
  float s = (upper ? v.y : v.x) + __shfl_xor_sync(0xFFFFFFFFu, upper ? v.x : v.y, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const float other = __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  return upper ? make_float2(other, s) : make_float2(s, other);
}

// Row groups of `nw` warps within a CTA, and their sums: every warp of the group gets the total.  Two
// buffers in turn, so that one barrier per sum is enough.
struct RowGroup {
  int nw, id, w;
  float2 *sh;   // 2 x 16
  int turn = 0;
  __device__ __forceinline__ RowGroup(int nw_, float2 (*shared)[2][16]) : nw(nw_) {
    const int warp = threadIdx.x >> 5;
    id = warp / nw;
    w = warp - id * nw;
    sh = &shared[id][0][0];
  }
  // every warp's v; lane k < nw gets warp k's, the others zeros
  __device__ __forceinline__ float2 share(float2 v) {
    const int lane = threadIdx.x & 31;
    float2 *b = sh + 16 * turn;
    turn ^= 1;
    if (lane == 0) b[w] = v;
    asm volatile("bar.sync %0, %1;\n" ::"r"(1 + id), "r"(32 * nw) : "memory");
    return lane < nw ? b[lane] : make_float2(0.0f, 0.0f);
  }
  __device__ __forceinline__ float2 sum(float2 v) {
    v = warp_sum2(v);
    if (nw == 1) return v;
    return warp_sum2(share(v));
  }
  // The row's mean and sum of squared deviations from the warps' (warp k holds `width` columns from
  // k width on, as far as the row goes).
  __device__ __forceinline__ float2 moments(float mean, float m2, int d, int width, float inv_d) {
    if (nw == 1) return make_float2(mean, m2);
    const float2 v = share(make_float2(mean, m2));
    const float n = (float)min(max(d - (int)(threadIdx.x & 31) * width, 0), width);
    const float m = warp_sum(v.x * n) * inv_d, dev = v.x - m;
    return make_float2(m, warp_sum(fmaf(n * dev, dev, v.y)));
  }
};

// C per-column factors of a lane (c0: the piece's first column)
template <bool VEC, int C = 16>
__device__ __forceinline__ void load_cols(const float *p, int c0, int n, int lane, float fill, float2 *v) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < C / 2; ++k) v[k] = both(fill);
  } else if (VEC) {
#pragma unroll
    for (int k = 0; k < C / 2; k += 2) {
      const float4 f = C * lane < n ? __ldg(reinterpret_cast<const float4 *>(p + c0 + C * lane + 2 * k))
                                    : make_float4(fill, fill, fill, fill);
      v[k] = make_float2(f.x, f.y);
      v[k + 1] = make_float2(f.z, f.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < C / 2; ++k) {
      const int c = 64 * k + lane;
      v[k] = make_float2(c < n ? __ldg(p + c0 + c) : fill, c + 32 < n ? __ldg(p + c0 + c + 32) : fill);
    }
  }
}
// v where the lane's pair k lies in the row, 0 elsewhere
template <bool VEC>
__device__ __forceinline__ float2 in_row2(int n, int lane, int k, float2 v) {
  if (VEC) return 16 * lane < n ? v : both(0.0f);
  return make_float2(64 * k + lane < n ? v.x : 0.0f, 64 * k + 32 + lane < n ? v.y : 0.0f);
}
__device__ __forceinline__ float sum2(float2 v) { return v.x + v.y; }
// Whether a row's statistics are numbers.  A variance that overflowed leaves rstd at 0, which is finite.
__device__ __forceinline__ bool norm_row_ok(float mean, float var, float rstd) {
  return isfinite(mean) && isfinite(var) && isfinite(rstd);
}

// Mean and squared deviations of a row: each warp's own by two passes over its registers, then the
// warps' joined (mean = sum n_w mean_w / d, M2 = sum M2_w + n_w (mean_w - mean)^2), so that no large
// mean is squared and the row group meets at one barrier only.  U = 1 holds gain and offset in
// registers, U = 2 and 3 in shared memory where no bank conflicts (8192 x 16384 BF16: 97 us, 179 with
// loads from L1 and L2, whose lines 32 lanes' 64 bytes each cross); both load the next row before they
// wait for the sums of this one (231 us without either).  U = 4 has room for neither.  The 80 registers of
// U = 1 (three CTAs per SM) spill 12 to 52 bytes.
template <typename E, bool VEC, int U, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? (U == 1 ? 3 : 2) : MAXT == 384 ? 2 : 1)
    k_norm_forward(const __grid_constant__ NormForward a, int nw, int fmt, int *status) {
  __shared__ float2 red[16][2][16];
  const int lane = threadIdx.x & 31, T = a.T, d = a.d, groups = (d + kActGroup - 1) / kActGroup;
  RowGroup G(nw, red);
  const int per_cta = (int)(blockDim.x >> 5) / nw, step = gridDim.x * per_cta;
  const int first = G.w * U * kPiece, mine = min(max(d - first, 0), U * kPiece);   // the warp's columns
  const float inv_d = __frcp_rn((float)d), inv_mine = mine ? __frcp_rn((float)mine) : 0.0f;
  float2 g[8], b[8];
  if (U == 1) {
    load_cols<VEC>(a.gamma, first, d - first, lane, 1.0f, g);
    load_cols<VEC>(a.beta, first, d - first, lane, 0.0f, b);
  }
  extern __shared__ float4 cols_sh[];
  float4 *const own = cols_sh + G.w * U * 2 * 128 + lane;   // [piece][gain, offset][4][32]: no bank conflicts
  if (U == 2 || U == 3) {
#pragma unroll
    for (int u = 0; u < U && G.id == 0; ++u) {
      load_cols<VEC>(a.gamma, first + u * kPiece, d - first - u * kPiece, lane, 1.0f, g);
      load_cols<VEC>(a.beta, first + u * kPiece, d - first - u * kPiece, lane, 0.0f, b);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        own[(8 * u + k) * 32] = make_float4(g[2 * k].x, g[2 * k].y, g[2 * k + 1].x, g[2 * k + 1].y);
        own[(8 * u + 4 + k) * 32] = make_float4(b[2 * k].x, b[2 * k].y, b[2 * k + 1].x, b[2 * k + 1].y);
      }
    }
    __syncthreads();
  }
  constexpr bool kAhead = U <= 3;
  Raw<E> now[U], next[kAhead ? U : 1];
  auto load = [&](int t, Raw<E> *r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c0 = first + u * kPiece;
      load_piece<VEC>(static_cast<const E *>(a.x) + (size_t)t * d + c0, t < T ? d - c0 : 0, lane, r[u]);
    }
  };
  int t = blockIdx.x * per_cta + G.id;
  if (kAhead) load(t, next);
  for (; t < T; t += step) {
    const size_t row = (size_t)t * d;
    if (kAhead) {
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = next[kAhead ? u : 0];
      load(t + step, next);
    } else {
      load(t, now);
    }
    float2 x[U][8], s = both(0.0f), q = both(0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[u][k] = now[u].pair(k);
        s = add2(s, x[u][k]);
      }
    const float wmean = warp_sum(sum2(s)) * inv_mine;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 v = in_row2<VEC>(d - first - u * kPiece, lane, k, add2(x[u][k], both(-wmean)));
        q = fma2(v, v, q);
      }
    const float2 st = G.moments(wmean, warp_sum(sum2(q)), d, U * kPiece, inv_d);
    const float mean = st.x, var = fmaf(st.y, inv_d, a.eps), rstd = __frcp_rn(__fsqrt_rn(var));
    if (G.w == 0 && lane == 0) {
      if (a.mean) a.mean[t] = mean;
      if (a.rstd) a.rstd[t] = rstd;
      if (!norm_row_ok(mean, var, rstd)) set_status(status, GIFT_ERR_NONFINITE);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c0 = first + u * kPiece, n = d - c0;
      if (n > 0) {
        if (U == 2 || U == 3) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 gv = own[(8 * u + k) * 32], bv = own[(8 * u + 4 + k) * 32];
            g[2 * k] = make_float2(gv.x, gv.y);
            g[2 * k + 1] = make_float2(gv.z, gv.w);
            b[2 * k] = make_float2(bv.x, bv.y);
            b[2 * k + 1] = make_float2(bv.z, bv.w);
          }
        } else if (U > 3) {
          load_cols<VEC>(a.gamma, c0, n, lane, 1.0f, g);
          load_cols<VEC>(a.beta, c0, n, lane, 0.0f, b);
        }
        float2 y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[u][k] = in_row2<VEC>(n, lane, k, mul2(add2(x[u][k], both(-mean)), both(rstd)));
          y[k] = fma2(x[u][k], g[k], b[k]);
        }
        store_piece<VEC>(static_cast<E *>(a.y) + row + c0, n, lane, y);
        if (a.codes) {
          uint8_t *cp = a.codes + row + c0, *sp = a.scales + (size_t)t * groups + c0 / kActGroup;
          if (fmt == FMT_E4M3) encode_piece<FMT_E4M3, VEC>(x[u], n, lane, cp, sp);
          else encode_piece<FMT_E5M2, VEC>(x[u], n, lane, cp, sp);
        }
      }
    }
  }
}

// What the backward pass needs of a lane's C columns of a row, as loaded.
template <typename E, bool SAVED, int C>
struct RowPiece {
  Raw<E, C> dy;
  Raw<E, C> x;
};
template <typename E, int C>
struct RowPiece<E, true, C> {
  Raw<E, C> dy;
  RawCodes<C> x;
};

template <int C>
constexpr int kColWords = C * 33;   // a warp's column sums in shared memory

// a lane's C column sums of a piece to out (n columns are left)
template <bool VEC, int C>
__device__ __forceinline__ void write_cols(float *out, int n, int lane, const float2 *v) {
#pragma unroll
  for (int e = 0; e < C; ++e) {
    const int c = piece_col<VEC, C>(lane, e);
    if (c < n) out[c] = e & 1 ? v[e / 2].y : v[e / 2].x;
  }
}

// U = 1 (up to 8192 columns): dx and the column sums.  The two sums, the gain and two rows take eight
// registers a column, so at most 16 warps per SM with C = 16 columns per lane (120 to 128 registers), 24
// with C = 8 up to 2048 columns (80); from 2049 to 4096 C = 8 takes 97 to 103 in CTAs of one row, 9 to 16
// warps per SM.  With 32-byte accesses C = 16 is faster (32768 x 4096 BF16: 171 us against 203; 16384
// x 1536 from the checkpoint 38 against 41), with element accesses C = 8 (5003 x 1361 FP32 from the
// checkpoint: 29 us against 37; 30324 x 20: 16 against 22).
// U > 1 (longer rows): dx alone, the column sums take a pass of their own (k_norm_cols).
// Spilled (bytes stored): FP32 with wide accesses 16, elements 8 to 96; U = 2 up to 40, U = 4 190 to 310.
template <typename E, bool VEC, bool SAVED, int U, int C, int MAXT>
__global__ void __launch_bounds__(MAXT, U > 1 || MAXT == 512 ? 1 : C == 16 ? 2 : 3)
    k_norm_backward(const __grid_constant__ NormBackward a, int nw, int fmt, int *status) {
  extern __shared__ float acc_sh[];
  __shared__ float2 red[16][2][16];
  grid_release();
  constexpr int kWide = 32 * C;   // columns of a piece
  const int lane = threadIdx.x & 31, T = a.T, d = a.d, groups = (d + kActGroup - 1) / kActGroup;
  RowGroup G(nw, red);
  const int per_cta = (int)(blockDim.x >> 5) / nw, step = gridDim.x * per_cta;
  const int first = G.w * U * kWide;
  const float inv_d = __frcp_rn((float)d);
  float2 g[C / 2], dg[C / 2], db[C / 2];   // U = 1: held for the CTA's rows
  if (U == 1) load_cols<VEC, C>(a.gamma, first, d - first, lane, 1.0f, g);
#pragma unroll
  for (int k = 0; k < C / 2; ++k) dg[k] = db[k] = both(0.0f);
  RowPiece<E, SAVED, C> now[U], next[1];
  auto load = [&](int t, RowPiece<E, SAVED, C> *p) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c0 = first + u * kWide, n = t < T ? d - c0 : 0;
      const size_t at = (size_t)t * d + c0;
      load_piece<VEC>(static_cast<const E *>(a.dy) + at, n, lane, p[u].dy);
      if constexpr (SAVED)
        load_codes<VEC>(a.codes + at, a.scales + (size_t)t * groups + c0 / kActGroup, n, lane, p[u].x);
      else
        load_piece<VEC>(static_cast<const E *>(a.x) + at, n, lane, p[u].x);
    }
  };
  int t = blockIdx.x * per_cta + G.id;
  if (U == 1) load(t, next);
  for (; t < T; t += step) {
    const float rstd = a.rstd[t], mean = SAVED ? 0.0f : a.mean[t];
    if (U == 1) {
      now[0] = next[0];
      load(t + step, next);
    } else {
      load(t, now);
    }
    auto n_of = [&](int u, int k) -> float2 {
      if constexpr (SAVED)
        return fmt == FMT_E4M3 ? code_pair<FMT_E4M3, VEC>(now[u].x, k) : code_pair<FMT_E5M2, VEC>(now[u].x, k);
      else
        return mul2(add2(now[u].x.pair(k), both(-mean)), both(rstd));
    };
    float2 sh = both(0.0f), shn = both(0.0f);
    float2 keep[C / 2];   // U = 1: n
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1) load_cols<VEC, C>(a.gamma, first + u * kWide, d - first - u * kWide, lane, 1.0f, g);
#pragma unroll
      for (int k = 0; k < C / 2; ++k) {
        const float2 dy = now[u].dy.pair(k), h = mul2(dy, g[k]), n = n_of(u, k);
        if (U == 1) {
          keep[k] = n;
          dg[k] = fma2(dy, n, dg[k]);
          db[k] = add2(db[k], dy);
        }
        sh = add2(sh, h);
        shn = fma2(h, n, shn);
      }
    }
    const float2 s = G.sum(make_float2(sum2(sh), sum2(shn)));
    if (G.w == 0 && lane == 0 && !(isfinite(s.x) && isfinite(s.y) && isfinite(rstd)))
      set_status(status, GIFT_ERR_NONFINITE);
    const float2 ma = both(-s.x * inv_d), mb = both(-s.y * inv_d);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c0 = first + u * kWide;
      if (U > 1) load_cols<VEC, C>(a.gamma, c0, d - c0, lane, 1.0f, g);
      float2 dx[C / 2];
#pragma unroll
      for (int k = 0; k < C / 2; ++k)
        dx[k] = mul2(both(rstd), fma2(U == 1 ? keep[k] : n_of(u, k), mb, fma2(now[u].dy.pair(k), g[k], ma)));
      store_piece<VEC, C>(static_cast<E *>(a.dx) + (size_t)t * d + c0, d - c0, lane, dx);
    }
  }
  if (U > 1 || !a.part) return;
  // The CTA's partial.  Several row groups: every warp leaves its sums in shared memory (a lane's columns
  // 33 words apart, so that neither the writes by lane nor the reads by column conflict), then each
  // thread adds the groups' values of its columns in order.
  float *out = a.part + (size_t)2 * blockIdx.x * d;
  if (per_cta == 1) {
    write_cols<VEC, C>(out + first, d - first, lane, dg);
    write_cols<VEC, C>(out + d + first, d - first, lane, db);
    return;
  }
  constexpr int kWords = kColWords<C>;
  float *mine = acc_sh + 2 * kWords * (G.id * nw + G.w);
#pragma unroll
  for (int e = 0; e < C; ++e) {
    mine[33 * e + lane] = e & 1 ? dg[e / 2].y : dg[e / 2].x;
    mine[kWords + 33 * e + lane] = e & 1 ? db[e / 2].y : db[e / 2].x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * d; i += blockDim.x) {
    const int c = i < d ? i : i - d, in = c % kWide;
    const int e = VEC ? in % C : in / 32, l = VEC ? in / C : in % 32;
    const float *p = acc_sh + 2 * kWords * (c / kWide) + (i < d ? 0 : kWords) + 33 * e + l;
    float v = p[0];
    for (int k = 1; k < per_cta; ++k) v += p[2 * kWords * nw * k];
    out[i] = v;
  }
}

// The column sums alone: a warp takes one piece of the columns over a slice of consecutive tokens;
// part[2 slice] = sum dy n, part[2 slice + 1] = sum dy.  It reads dy and x a second time: 8192 x 16384 BF16
// take 200 us for dx (4.0 TB/s; no row is loaded ahead) and 124 us here (4.3 TB/s), 324 of a floor of 119.
template <typename E, bool VEC, bool SAVED>
__global__ void __launch_bounds__(kNormThreads) k_norm_cols(const __grid_constant__ NormBackward a, int fmt, int rows) {
  const int lane = threadIdx.x & 31, d = a.d, groups = (d + kActGroup - 1) / kActGroup;
  const int c0 = (blockIdx.x * (kNormThreads / 32) + (threadIdx.x >> 5)) * kPiece, n = d - c0;
  grid_release();
  if (n <= 0) return;
  float2 dg[8], db[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) dg[k] = db[k] = both(0.0f);
  const int t1 = min(a.T, (int)(blockIdx.y + 1) * rows);
#pragma unroll 2
  for (int t = blockIdx.y * rows; t < t1; ++t) {
    const size_t at = (size_t)t * d + c0;
    RowPiece<E, SAVED, 16> p;
    load_piece<VEC>(static_cast<const E *>(a.dy) + at, n, lane, p.dy);
    float rstd = 1.0f, mean = 0.0f;
    if constexpr (SAVED) {
      load_codes<VEC>(a.codes + at, a.scales + (size_t)t * groups + c0 / kActGroup, n, lane, p.x);
    } else {
      load_piece<VEC>(static_cast<const E *>(a.x) + at, n, lane, p.x);
      rstd = a.rstd[t];
      mean = a.mean[t];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 dy = p.dy.pair(k);
      float2 v;
      if constexpr (SAVED) v = fmt == FMT_E4M3 ? code_pair<FMT_E4M3, VEC>(p.x, k) : code_pair<FMT_E5M2, VEC>(p.x, k);
      else v = mul2(add2(p.x.pair(k), both(-mean)), both(rstd));
      dg[k] = fma2(dy, v, dg[k]);
      db[k] = add2(db[k], dy);
    }
  }
  float *out = a.part + (size_t)2 * blockIdx.y * d;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int c = c0 + piece_col<VEC>(lane, e);
    if (c < d) {
      out[c] = e & 1 ? dg[e / 2].y : dg[e / 2].x;
      out[d + c] = e & 1 ? db[e / 2].y : db[e / 2].x;
    }
  }
}

// out[c] = sum over partials of part[k stride + c]: 32 columns per CTA, 32 warps take every 32nd
// partial (their loads are all in flight at once: latency is what this kernel costs, 5 us for 152
// partials of 2 x 1536 columns), and their sums are added in order.  blockIdx.y: the first or the second output.
__global__ void __launch_bounds__(1024) k_norm_sums(const float *__restrict__ part, int parts, size_t stride,
                                                    size_t second, int d, float *out0, float *out1) {
  __shared__ float sh[32][33];
  grid_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float *out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const float *p = part + blockIdx.y * second + c;
  float s = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int k = w; k < parts; k += 32) s += p[k * stride];
  }
  sh[w][lane] = s;
  __syncthreads();
  const float v = warp_sum(sh[lane][w]);   // column w of the block
  if (lane == 0 && blockIdx.x * 32 + w < d) out[blockIdx.x * 32 + w] = v;
}

// ---- rows too long for registers: column by column, the row read once per sum --------------------------
// (above 32768 columns.)  A row is read three times forward and twice backward, L2 serves the repeats:
// 4096 x 40960 BF16 287 us forward, 863 us backward with both sums over tokens, 1046 from the checkpoint.
__device__ __forceinline__ float cta_sum(float v, float *sh /* kNormThreads / 32 */) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) r += sh[i];
  return r;
}

template <typename E>
__global__ void __launch_bounds__(kNormThreads) k_norm_forward_long(const __grid_constant__ NormForward a, int fmt,
                                                                    int *status) {
  __shared__ float sh[kNormThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = a.d;
  const int groups = (d + kActGroup - 1) / kActGroup;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = (size_t)t * d;
    const E *xr = static_cast<const E *>(a.x) + row;
    float s = 0.0f;
    for (int c = threadIdx.x; c < d; c += kNormThreads) s += ld1(xr + c);
    const float mean = __fdiv_rn(cta_sum(s, sh), (float)d);
    float q = 0.0f;
    for (int c = threadIdx.x; c < d; c += kNormThreads) {
      const float u = ld1(xr + c) - mean;
      q = fmaf(u, u, q);
    }
    const float var = __fdiv_rn(cta_sum(q, sh), (float)d) + a.eps, rstd = __frcp_rn(__fsqrt_rn(var));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[t] = mean;
      if (a.rstd) a.rstd[t] = rstd;
      if (!norm_row_ok(mean, var, rstd)) set_status(status, GIFT_ERR_NONFINITE);
    }
    for (int c0 = warp * kPiece; c0 < d; c0 += kNormThreads / 32 * kPiece) {
      const int n = d - c0;
      Raw<E> r;
      load_piece<false>(xr + c0, n, lane, r);
      float2 x[8], g[8], b[8], y[8];
      load_cols<false>(a.gamma, c0, n, lane, 1.0f, g);
      load_cols<false>(a.beta, c0, n, lane, 0.0f, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = in_row2<false>(n, lane, k, mul2(add2(r.pair(k), both(-mean)), both(rstd)));
        y[k] = fma2(x[k], g[k], b[k]);
      }
      store_piece<false>(static_cast<E *>(a.y) + row + c0, n, lane, y);
      if (a.codes) {
        uint8_t *cp = a.codes + row + c0, *sp = a.scales + (size_t)t * groups + c0 / kActGroup;
        if (fmt == FMT_E4M3) encode_piece<FMT_E4M3, false>(x, n, lane, cp, sp);
        else encode_piece<FMT_E5M2, false>(x, n, lane, cp, sp);
      }
    }
  }
}

// The normalised element (t, c) from what the forward pass kept.
template <typename E>
__device__ __forceinline__ float saved_at(const NormBackward &a, int fmt, int groups, int t, int c) {
  const size_t i = (size_t)t * a.d + c;
  if (a.codes) {
    const float s = act_scale(a.scales[(size_t)t * groups + c / kActGroup]);
    return (fmt == FMT_E4M3 ? dec_e4m3(a.codes[i]) : dec_e5m2(a.codes[i])) * s;
  }
  return (ld1(static_cast<const E *>(a.x) + i) - a.mean[t]) * a.rstd[t];
}

template <typename E>
__global__ void __launch_bounds__(kNormThreads) k_norm_dx_long(const __grid_constant__ NormBackward A, int fmt,
                                                               int *status) {
  __shared__ float sh[kNormThreads / 32];
  const int d = A.d, groups = (d + kActGroup - 1) / kActGroup;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    const E *dy = static_cast<const E *>(A.dy) + (size_t)t * d;
    float a = 0.0f, b = 0.0f;
    for (int c = threadIdx.x; c < d; c += kNormThreads) {
      const float h = ld1(dy + c) * (A.gamma ? A.gamma[c] : 1.0f);
      a += h;
      b = fmaf(h, saved_at<E>(A, fmt, groups, t, c), b);
    }
    a = __fdiv_rn(cta_sum(a, sh), (float)d);
    b = __fdiv_rn(cta_sum(b, sh), (float)d);
    const float rstd = A.rstd[t];
    if (threadIdx.x == 0 && !(isfinite(a) && isfinite(b) && isfinite(rstd))) set_status(status, GIFT_ERR_NONFINITE);
    for (int c = threadIdx.x; c < d; c += kNormThreads) {
      const float h = ld1(dy + c) * (A.gamma ? A.gamma[c] : 1.0f);
      st1(static_cast<E *>(A.dx) + (size_t)t * d + c, rstd * (h - a - saved_at<E>(A, fmt, groups, t, c) * b));
    }
  }
}

// ---- host ---------------------------------------------------------------------------------------------
// tokens of a slice of a column pass: at least 16, at most 256 slices
int col_rows(int T) {
  const int r = (T + 255) / 256;
  return r < 16 ? 16 : r;
}

bool cols_aligned(const float *p) { return !p || aligned16(p); }

// CTAs of a persistent launch: what is resident on the context's SMs, at most one per `per_cta` rows.
template <auto Kernel>
int resident(const Launch &L, int threads, int smem, int T, int per_cta) {
  const long long most = (long long)L.sms * resident_per_sm<Kernel>(threads, smem);
  const long long need = ((long long)T + per_cta - 1) / per_cta;
  return (int)(need < most ? need : most);
}

// Rows by registers: pieces per lane and warps per row.
struct RowPlan {
  int u, nw, threads;
  int c = 16;   // columns per lane
};

// CTAs of whole row groups, about eight warps
int group_threads(int nw) { return 32 * nw * (nw >= 8 ? 1 : 8 / nw); }

// As many warps per row as pieces up to 8192 columns, then two or four pieces per lane; CTAs of 8 to
// 16 warps.
bool row_plan(int d, RowPlan *p) {
  const int pieces = (d + kPiece - 1) / kPiece;
  if (pieces > 64) return false;
  p->u = pieces <= 16 ? 1 : pieces <= 32 ? 2 : 4;
  p->nw = (pieces + p->u - 1) / p->u;
  p->threads = group_threads(p->nw);
  return true;
}

// Backward: element accesses up to 4096 columns by 256 columns and warp, else as the forward pass; where
// the warps of a row do not divide eight, all the row groups that 16 warps hold in one CTA (three
// warps per row: 15 warps per SM instead of 12).
bool backward_plan(int d, bool vec, RowPlan *p) {
  if (!vec && d <= 16 * 256) {
    p->u = 1;
    p->c = 8;
    p->nw = (d + 255) / 256;
    p->threads = group_threads(p->nw);
    return true;
  }
  if (!row_plan(d, p)) return false;
  if (p->u == 1 && p->nw < 8 && 8 % p->nw) p->threads = 32 * p->nw * (16 / p->nw);
  return true;
}

// Forward: with 32-byte accesses two pieces per lane where that leaves at most a sixth of the lanes idle (fewer
// warps to a row, twice the loads of a lane in flight: 32768 x 4096 BF16 91 us against 101, 111 against
// 131 with the checkpoint; 8192 x 8192 52 against 62), and a whole row of three pieces in one BF16 warp,
// which needs no barrier (16384 x 1536: 20.3 against 22.8, 26.8 against 28.9; also where the third piece is
// mostly empty, 32768 rows of 1040 columns 35.5 against 41.6, 45.7 against 51.8, of 1280 35.5 against
// 41.6, 45.7 against 53.9; FP32 would not fit the registers).  With element accesses one piece was faster
// (4099 x 7001 BF16 72 us against 87).
bool forward_plan(int d, bool vec, bool bf16, RowPlan *p) {
  if (!row_plan(d, p)) return false;
  const int pieces = (d + kPiece - 1) / kPiece;
  if (!vec || p->u > 1 || pieces == 1) return true;
  if (pieces == 3 && bf16) {
    p->u = 3;
    p->nw = 1;
    p->threads = 256;
  } else if (pieces % 2 == 0 || pieces >= 5) {
    p->u = 2;
    p->nw = (pieces + 1) / 2;
    p->threads = group_threads(p->nw);
  }
  return true;
}

template <typename E, bool VEC, int U, int MAXT>
cudaError_t forward_t(const Launch &L, int fmt, const NormForward &a, const RowPlan &p) {
  constexpr auto kernel = k_norm_forward<E, VEC, U, MAXT>;
  const int smem = U == 2 || U == 3 ? p.nw * U * 2 * kPiece * (int)sizeof(float) : 0;   // gain and offset
  if (smem) {
    const cudaError_t e = ensure_dynamic_smem<kernel>(16 * U * 2 * kPiece * (int)sizeof(float));
    if (e != cudaSuccess) return e;
  }
  kernel<<<resident<kernel>(L, p.threads, smem, a.T, p.threads / 32 / p.nw), p.threads, smem, L.stream>>>(
      a, p.nw, fmt, L.status);
  return cudaGetLastError();
}

// The CTA sizes that forward_plan gives: one piece, 8 warps at most with wide accesses and up to 16 with
// element ones; two pieces, 8 warps for 5 to 16 pieces (wide) and 9 to 16 warps above; four pieces, 9 to 16.
template <typename E, bool VEC, int U>
cudaError_t forward(const Launch &L, int fmt, const NormForward &a, const RowPlan &p) {
  if constexpr (VEC && U == 1) {
    return forward_t<E, VEC, U, 256>(L, fmt, a, p);
  } else {
    if constexpr (U == 1 || (VEC && U == 2))
      if (p.threads <= 256) return forward_t<E, VEC, U, 256>(L, fmt, a, p);
    if constexpr (U == 1)
      if (p.threads <= 384) return forward_t<E, VEC, U, 384>(L, fmt, a, p);
    return forward_t<E, VEC, U, 512>(L, fmt, a, p);
  }
}

template <typename E, bool VEC>
cudaError_t forward_u(const Launch &L, int fmt, const NormForward &a, const RowPlan &p) {
  if constexpr (VEC && sizeof(E) == 2)
    if (p.u == 3) return forward_t<E, VEC, 3, 256>(L, fmt, a, p);
  switch (p.u) {
    case 1: return forward<E, VEC, 1>(L, fmt, a, p);
    case 2: return forward<E, VEC, 2>(L, fmt, a, p);
    default: return forward<E, VEC, 4>(L, fmt, a, p);
  }
}

template <typename E>
cudaError_t forward_e(const Launch &L, int fmt, const NormForward &a) {
  RowPlan p;
  const bool vec = rows_vec(a.d, a.x, a.codes) && rows_vec(a.d, a.y, nullptr) && cols_aligned(a.gamma) &&
                   cols_aligned(a.beta);
  if (!forward_plan(a.d, vec, sizeof(E) == 2, &p)) {
    const int grid = a.T < L.sms * 8 ? a.T : L.sms * 8;
    k_norm_forward_long<E><<<grid, kNormThreads, 0, L.stream>>>(a, fmt, L.status);
    return cudaGetLastError();
  }
  return vec ? forward_u<E, true>(L, fmt, a, p) : forward_u<E, false>(L, fmt, a, p);
}

cudaError_t sums_after(const Launch &L, const NormBackward &a, int parts) {
  return launch_after(L.stream, k_norm_sums, dim3((a.d + 31) / 32, 2), 1024, a.part, parts, (size_t)2 * a.d,
                      (size_t)a.d, a.d, a.dgamma, a.dbeta);
}

template <typename E, bool VEC, bool SAVED>
cudaError_t column_pass(const Launch &L, int fmt, const NormBackward &a) {
  if (!a.part) return cudaSuccess;
  const int rows = col_rows(a.T), slices = (a.T + rows - 1) / rows, per = kNormThreads / 32 * kPiece;
  k_norm_cols<E, VEC, SAVED><<<dim3((a.d + per - 1) / per, slices), kNormThreads, 0, L.stream>>>(a, fmt, rows);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : sums_after(L, a, slices);
}

template <typename E, bool VEC, bool SAVED, int U, int C, int MAXT>
cudaError_t backward_t(const Launch &L, int fmt, const NormBackward &a, const RowPlan &p) {
  constexpr auto kernel = k_norm_backward<E, VEC, SAVED, U, C, MAXT>;
  const int warps = p.threads / 32, per_cta = warps / p.nw, smem = U == 1 && per_cta > 1 ? warps * 2 * kColWords<C> * 4 : 0;
  cudaError_t e = smem ? ensure_dynamic_smem<kernel>(MAXT / 32 * 2 * kColWords<C> * 4) : cudaSuccess;
  if (e != cudaSuccess) return e;
  int grid = resident<kernel>(L, p.threads, smem, a.T, per_cta);
  if (grid > norm_partials(L.sms, a.T)) grid = norm_partials(L.sms, a.T);
  kernel<<<grid, p.threads, smem, L.stream>>>(a, p.nw, fmt, L.status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (U > 1) return column_pass<E, VEC, SAVED>(L, fmt, a);
  return a.part ? sums_after(L, a, grid) : cudaSuccess;
}

// The CTA sizes that backward_plan gives: 8 columns per lane for element accesses up to 4096 columns; 16
// elsewhere, in 9 to 16 warps but for wide accesses to up to 8 pieces.
template <typename E, bool VEC, bool SAVED, int U>
cudaError_t backward(const Launch &L, int fmt, const NormBackward &a, const RowPlan &p) {
  if constexpr (U == 1) {
    constexpr int kSmall = VEC ? 16 : 8;   // columns per lane of the CTAs of 256 threads
    if (p.threads <= 256) return backward_t<E, VEC, SAVED, U, kSmall, 256>(L, fmt, a, p);
    if constexpr (!VEC)
      if (p.c == 8) return backward_t<E, VEC, SAVED, U, 8, 512>(L, fmt, a, p);
  }
  return backward_t<E, VEC, SAVED, U, 16, 512>(L, fmt, a, p);
}

template <typename E, bool VEC, bool SAVED>
cudaError_t backward_s(const Launch &L, int fmt, const NormBackward &a) {
  RowPlan p;
  if (backward_plan(a.d, VEC, &p)) {
    switch (p.u) {
      case 1: return backward<E, VEC, SAVED, 1>(L, fmt, a, p);
      case 2: return backward<E, VEC, SAVED, 2>(L, fmt, a, p);
      default: return backward<E, VEC, SAVED, 4>(L, fmt, a, p);
    }
  }
  const int grid = a.T < L.sms * 8 ? a.T : L.sms * 8;
  k_norm_dx_long<E><<<grid, kNormThreads, 0, L.stream>>>(a, fmt, L.status);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : column_pass<E, VEC, SAVED>(L, fmt, a);
}

template <typename E>
cudaError_t backward_e(const Launch &L, int fmt, const NormBackward &a) {
  const bool vec = rows_vec(a.d, a.dy, a.codes) && rows_vec(a.d, a.dx, nullptr) && rows_vec(a.d, a.x, nullptr) &&
                   cols_aligned(a.gamma);
  if (a.codes) return vec ? backward_s<E, true, true>(L, fmt, a) : backward_s<E, false, true>(L, fmt, a);
  return vec ? backward_s<E, true, false>(L, fmt, a) : backward_s<E, false, false>(L, fmt, a);
}

}  // namespace

// partials of the backward pass: a CTA each, at most four per SM
int norm_partials(int sms, int T) {
  const long long most = (long long)sms * 4;
  return (int)(T < most ? T : most);
}

size_t norm_part_floats(int sms, int T, int d) {
  RowPlan p;
  if (row_plan(d, &p) && p.u == 1) return (size_t)2 * norm_partials(sms, T) * d;
  const int rows = col_rows(T);
  return (size_t)2 * ((T + rows - 1) / rows) * d;
}

cudaError_t launch_norm_forward(const Launch &L, int fmt, bool bf16, const NormForward &a) {
  return bf16 ? forward_e<__nv_bfloat16>(L, fmt, a) : forward_e<float>(L, fmt, a);
}

cudaError_t launch_norm_backward(const Launch &L, int fmt, bool bf16, const NormBackward &a) {
  return bf16 ? backward_e<__nv_bfloat16>(L, fmt, a) : backward_e<float>(L, fmt, a);
}

cudaError_t launch_sum_parts(const Launch &L, const float *part, int parts, int d, float *out) {
  return launch_after(L.stream, k_norm_sums, dim3((d + 31) / 32, 1), 1024, part, parts, (size_t)d, (size_t)0, d, out,
                      static_cast<float *>(nullptr));
}

}  // namespace gift
