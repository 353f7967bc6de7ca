// Operands of the tensor-core products as their TMA loads want them: rows at a 16-byte pitch, and FP32 as
// three BF16 terms.  Device functions that walk a matrix with a part of a launch's CTAs (256 threads each).
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace gift {

// The terms of one value at the end of FP32's range, where rounding to BF16 gives an infinity.  A finite
// value is cut into its bits instead (8 + 8 + 8 of them, exact), so that no sum of the first terms passes it; an
// infinity or NaN is its own first term and has no others (Inf - Inf would make it NaN).
__device__ __forceinline__ void bf16_terms_of_large(float x, uint16_t *t) {
  const uint32_t bits = __float_as_uint(x), size = bits & 0x7FFFFFFFu;
  if (size < 0x7F7F8000u) {
    tc::bf16_split3(x, t[0], t[1], t[2]);
  } else if (size < 0x7F800000u) {
    const float r = __fsub_rn(x, __uint_as_float(bits & 0xFFFF0000u));
    t[0] = (uint16_t)(bits >> 16);
    t[1] = (uint16_t)(__float_as_uint(r) >> 16);
    t[2] = __bfloat16_as_ushort(__float2bfloat16_rn(__fsub_rn(r, __uint_as_float(__float_as_uint(r) & 0xFFFF0000u))));
  } else {
    t[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    t[1] = t[2] = 0;
  }
}

// Rows are cut into spans, so that a few long rows (the last tokens of a batch) keep many warps busy.
constexpr int kSpan = 1024;   // elements of BF16 terms
__host__ __device__ inline size_t spans(int T, size_t len, size_t span) { return (size_t)T * ((len + span - 1) / span); }

// FP32 as three BF16 terms (exact from 2^-110 up; below, the last ends at BF16's smallest step), planes of
// T rows of ld columns; a warp per span, two columns per lane
__device__ __forceinline__ void bf16_terms(const float *x, int T, int d, int ld, uint16_t *out, int cta, int ctas) {
  const size_t plane = (size_t)T * ld, all = spans(T, d, kSpan);
  const unsigned per = ((unsigned)d + kSpan - 1) / kSpan;
  for (size_t i = (size_t)cta * 8 + (threadIdx.x >> 5); i < all; i += (size_t)ctas * 8) {
    const size_t t = i / per;
    const int c0 = (int)(i - t * per) * kSpan, c1 = min(d, c0 + kSpan);
    const float *p = x + t * d;
    uint16_t *o = out + t * ld;
    for (int c = c0 + 2 * (threadIdx.x & 31); c < c1; c += 256) {   // ld and kSpan are even
      float v[4][2];   // all loads before the first store
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u][0] = c + 64 * u < c1 ? p[c + 64 * u] : 0.0f;
        v[u][1] = c + 64 * u + 1 < c1 ? p[c + 64 * u + 1] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (c + 64 * u >= c1) break;
        uint32_t w[3];
        const float x0 = v[u][0], x1 = v[u][1];
        if (max(abs_bits(x0), abs_bits(x1)) < 0x7F7F8000u) {
          tc::bf16_split3x2(x0, x1, w[0], w[1], w[2]);
        } else {
          uint16_t a[3], b[3];
          bf16_terms_of_large(x0, a);
          bf16_terms_of_large(x1, b);
#pragma unroll
          for (int k = 0; k < 3; ++k) w[k] = (uint32_t)a[k] | (uint32_t)b[k] << 16;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t *>(o + k * plane + c + 64 * u) = w[k];
      }
    }
  }
}

// 16 bytes that start `off` bytes into a, of the 32 in a and b
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  const int sh = 8 * (off & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                    __funnelshift_r(w[3], w[4], sh));
}
// the 16-byte block at p, zeros outside [lo, hi)
__device__ __forceinline__ uint4 aligned_block(uintptr_t p, uintptr_t lo, uintptr_t hi) {
  if (p >= lo && p + 16 <= hi) return *reinterpret_cast<const uint4 *>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};   // the ends of the matrix
#pragma unroll
  for (int b = 0; b < 16; ++b)
    if (p + b >= lo && p + b < hi) w[b / 4] |= (uint32_t)*reinterpret_cast<const uint8_t *>(p + b) << (8 * (b % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Rows of `bytes` bytes at any alignment -> rows of ld (a multiple of 16) bytes; a warp per span, 16 bytes
// per lane from the two aligned blocks that hold them.  Past a row's end nothing is read again (the
// tensor map's width).
__device__ __forceinline__ void repitch(const uint8_t *src, int T, size_t bytes, size_t ld, uint8_t *dst, int cta,
                                        int ctas) {
  constexpr size_t span = 2 * kSpan;
  const uintptr_t lo = (uintptr_t)src, hi = lo + (size_t)T * bytes;
  const size_t all = spans(T, bytes, span), per = (bytes + span - 1) / span;
  for (size_t i = (size_t)cta * 8 + (threadIdx.x >> 5); i < all; i += (size_t)ctas * 8) {
    const size_t t = i / per, c0 = (i - t * per) * span, c1 = min(bytes, c0 + span);
    const uintptr_t row = lo + t * bytes;
    const int off = (int)(row & 15);
    // Away from the matrix's ends every block is whole: all loads before the first store
    const bool inside = row + c0 - off >= lo && row + c1 + 32 <= hi;
    const size_t c = c0 + 16 * (threadIdx.x & 31);
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uintptr_t at = row + c + 512 * u - off;
      if (c + 512 * u >= c1) break;
      if (inside) {
        a[u] = *reinterpret_cast<const uint4 *>(at);
        b[u] = *reinterpret_cast<const uint4 *>(at + (off ? 16 : 0));
      } else {
        a[u] = aligned_block(at, lo, hi);
        b[u] = off ? aligned_block(at + 16, lo, hi) : a[u];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (c + 512 * u >= c1) break;
      *reinterpret_cast<uint4 *>(dst + t * ld + c + 512 * u) = shifted(a[u], b[u], off);
    }
  }
}

inline size_t pad16(size_t bytes) { return (bytes + 15) / 16 * 16; }

}  // namespace gift
