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
// 2^-k, what an element is multiplied with before it is rounded (k in [-110, 119]: normal); 1 for a
// marked group, whose codes mean nothing
__device__ __forceinline__ float act_inv_scale(uint32_t byte) {
  return byte == kActBad ? 1.0f : __uint_as_float((254u - byte) << 23);
}
// 2^k; NaN for a marked group
__device__ __forceinline__ float act_scale(uint32_t byte) {
  return byte == kActBad ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float ld1(const float *p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float *p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------------------------------------------
// Row pieces.  A warp handles a row in pieces of 32 C columns, C = 16 or 8 per lane, so that a piece
// holds whole scale groups.  Two layouts: VEC, for rows whose pitch and base allow 32-byte accesses
// (d a multiple of 16), lane l holds columns C l .. C l + C - 1 (a group is 128 / C lanes); otherwise
// lane l holds columns l, l + 32, ... (a group is four consecutive registers of the warp), each
// access one element wide and consecutive over the warp.
// ------------------------------------------------------------------------------------------------
constexpr int kPiece = 512;   // C = 16

__device__ __forceinline__ void ld256(const void *p, uint32_t *r) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void ld128(const void *p, uint32_t *r) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "l"(p));
}
__device__ __forceinline__ void st256(void *p, const uint32_t *r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two FP32 operations at once, each rounded to nearest.
__device__ __forceinline__ uint64_t as_b64(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 as_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_b64(a)), "l"(as_b64(b)));
  return as_f32x2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_b64(a)), "l"(as_b64(b)));
  return as_f32x2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_b64(a)), "l"(as_b64(b)), "l"(as_b64(c)));
  return as_f32x2(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The element type's registers for a lane's C columns of a piece, as loaded.
template <typename E, int C = 16>
struct Raw;
template <int C>
struct Raw<float, C> {
  uint32_t r[C];
  __device__ __forceinline__ float2 pair(int k) const {   // elements 2 k and 2 k + 1
    return make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
  }
};
template <int C>
struct Raw<__nv_bfloat16, C> {
  uint32_t r[C / 2];
  __device__ __forceinline__ float2 pair(int k) const {
    return make_float2(__uint_as_float(r[k] << 16), __uint_as_float(r[k] & 0xFFFF0000u));
  }
};

// column of a lane's e-th value within its piece
template <bool VEC, int C = 16>
__device__ __forceinline__ int piece_col(int lane, int e) { return VEC ? C * lane + e : 32 * e + lane; }

// Load a lane's values of the piece at p (n columns of the row are left, zeros past them).
template <bool VEC, int C>
__device__ __forceinline__ void load_piece(const float *p, int n, int lane, Raw<float, C> &x) {
  if (VEC) {
    if (C * lane < n) {
#pragma unroll
      for (int e = 0; e < C; e += 8) ld256(p + C * lane + e, x.r + e);
    } else {
#pragma unroll
      for (int e = 0; e < C; ++e) x.r[e] = 0u;
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e) x.r[e] = 32 * e + lane < n ? __float_as_uint(p[32 * e + lane]) : 0u;
  }
}
template <bool VEC, int C>
__device__ __forceinline__ void load_piece(const __nv_bfloat16 *p, int n, int lane, Raw<__nv_bfloat16, C> &x) {
  if (VEC) {
    if (C * lane < n) {
      if constexpr (C == 16) ld256(p + C * lane, x.r);
      else ld128(p + C * lane, x.r);
    } else {
#pragma unroll
      for (int e = 0; e < C / 2; ++e) x.r[e] = 0u;
    }
  } else {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
    uint32_t v[C];
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = 32 * e + lane < n ? (uint32_t)q[32 * e + lane] : 0u;
#pragma unroll
    for (int e = 0; e < C / 2; ++e) x.r[e] = v[2 * e] | v[2 * e + 1] << 16;
  }
}

template <bool VEC, int C = 16>
__device__ __forceinline__ void store_piece(float *p, int n, int lane, const float2 *v) {
  if (VEC) {
    if (C * lane < n) {
      uint32_t r[C];
#pragma unroll
      for (int k = 0; k < C / 2; ++k) {
        r[2 * k] = __float_as_uint(v[k].x);
        r[2 * k + 1] = __float_as_uint(v[k].y);
      }
#pragma unroll
      for (int e = 0; e < C; e += 8) st256(p + C * lane + e, r + e);
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (32 * e + lane < n) p[32 * e + lane] = e & 1 ? v[e / 2].y : v[e / 2].x;
  }
}
template <bool VEC, int C = 16>
__device__ __forceinline__ void store_piece(__nv_bfloat16 *p, int n, int lane, const float2 *v) {
  if (VEC) {
    if (C * lane < n) {
      uint32_t r[C / 2];
#pragma unroll
      for (int k = 0; k < C / 2; ++k) r[k] = pack_bf16(v[k].x, v[k].y);
      if constexpr (C == 16) st256(p + C * lane, r);
      else *reinterpret_cast<uint4 *>(p + C * lane) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (32 * e + lane < n) p[32 * e + lane] = __float2bfloat16_rn(e & 1 ? v[e / 2].y : v[e / 2].x);
  }
}

// Encode a lane's 16 values: codes to cp, the piece's scale bytes to sp.  Returns whether a group was
// marked.  All lanes of the warp call it.
template <int F, bool VEC>
__device__ __forceinline__ bool encode_piece(const float2 *v, int n, int lane, uint8_t *cp, uint8_t *sp) {
  if (VEC) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, max(abs_bits(v[k].x), abs_bits(v[k].y)));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const uint32_t sb = act_scale_byte<F>(m);
    const float2 inv = both(act_inv_scale(sb));
    if (16 * lane < n) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = mul2(v[2 * k], inv), b = mul2(v[2 * k + 1], inv);
        w[k] = pack4_fp8<F>(a.x, a.y, b.x, b.y);
      }
      *reinterpret_cast<uint4 *>(cp + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
      if ((lane & 7) == 0) sp[lane >> 3] = (uint8_t)sb;
    }
    return sb == kActBad;
  }
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = v[2 * k], b = v[2 * k + 1];
    const uint32_t sb = act_scale_byte<F>(
        warp_max_u32(max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(b.x), abs_bits(b.y)))));
    const float inv = act_inv_scale(sb);
    bad |= sb == kActBad;
    const uint32_t w = pack4_fp8<F>(__fmul_rn(a.x, inv), __fmul_rn(a.y, inv), __fmul_rn(b.x, inv), __fmul_rn(b.y, inv));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (32 * (4 * k + e) + lane < n) cp[32 * (4 * k + e) + lane] = (uint8_t)(w >> (8 * e));
    if (lane == 0 && kActGroup * k < n) sp[k] = (uint8_t)sb;
  }
  return bad;
}

// A lane's C codes of a piece and their scales, as loaded.
template <int C = 16>
struct RawCodes {
  uint32_t c[C / 4];   // VEC: the bytes in order; otherwise byte k of c[g] is element 4 g + k
  uint32_t s;          // VEC: the lane's scale byte; otherwise the groups' bytes
};
template <bool VEC, int C>
__device__ __forceinline__ void load_codes(const uint8_t *cp, const uint8_t *sp, int n, int lane, RawCodes<C> &x) {
  if (VEC) {
#pragma unroll
    for (int k = 0; k < C / 4; ++k) x.c[k] = 0u;
    x.s = 127u;
    if (C * lane < n) {
      if constexpr (C == 16) ld128(cp + C * lane, x.c);
      else asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(x.c[0]), "=r"(x.c[1]) : "l"(cp + C * lane));
      x.s = sp[lane * C / kActGroup];
    }
  } else {
    uint32_t mine = 127u;
    if (lane < C / 4 && kActGroup * lane < n) mine = sp[lane];
    x.s = 0;
#pragma unroll
    for (int g = 0; g < C / 4; ++g) {
      x.s |= __shfl_sync(0xFFFFFFFFu, mine, g) << (8 * g);
      x.c[g] = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (32 * (4 * g + k) + lane < n) x.c[g] |= (uint32_t)cp[32 * (4 * g + k) + lane] << (8 * k);
    }
  }
}
// The values of elements 2 k and 2 k + 1 (of one group in either layout): the hardware's conversion to
// FP16 holds every code exactly, and so does FP32.
template <int F, bool VEC, int C>
__device__ __forceinline__ float2 code_pair(const RawCodes<C> &x, int k) {
  const uint16_t c = (uint16_t)(k & 1 ? x.c[k >> 1] >> 16 : x.c[k >> 1] & 0xFFFFu);
  uint32_t h;
  if (F == FMT_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
  float2 v;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return mul2(v, both(act_scale(VEC ? x.s : (x.s >> (8 * (k >> 1))) & 0xFFu)));
}

// Walks the row pieces of a T x (pieces per row) grid in steps of a fixed number of warps, without a
// division per step.
struct PieceWalk {
  int t, p;
  int dt, dp, per;
  __device__ __forceinline__ PieceWalk(size_t first, size_t step, int per_row) : per(per_row) {
    t = (int)(first / per_row);
    p = (int)(first - (size_t)t * per_row);
    dt = (int)(step / per_row);
    dp = (int)(step - (size_t)dt * per_row);
  }
  __device__ __forceinline__ void next() {
    t += dt;
    p += dp;
    if (p >= per) {
      p -= per;
      ++t;
    }
  }
};

// Whether rows of d elements at x (32-byte accesses) and of d codes (16-byte) take the VEC layout.
inline bool rows_vec(int d, const void *x, const void *codes) {
  return d % 16 == 0 && ((uintptr_t)x & 31u) == 0 && ((uintptr_t)codes & 15u) == 0;
}

// wait for the programmatic predecessor's results / let the successor launch
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// launch with the programmatic dependency that grid_wait() ends
template <typename... P, typename... Q>
inline cudaError_t launch_after(cudaStream_t s, void (*kernel)(P...), dim3 grid, int threads, Q... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace gift
