// The 8-bit activation checkpoint: encode and decode.
//
// A warp takes a piece of 512 consecutive columns of one token (four scale groups) at a time: the
// groups' amax by shuffles, the scale exponent from the amax's bit pattern, the codes x 2^-k by the
// hardware's round-to-nearest-even, saturating conversion.  Both directions move each byte once
// (2 + 1 + 1/128 bytes an element for BF16) and HBM bounds them: 32-byte accesses, and enough warps
// that the next pieces' loads are in flight while one is converted.  16384 x 6144 BF16: encode 54.5 us,
// 5.5 TB/s; decode 53.8 us, 5.6 TB/s, 0.82 of the copy rate; 16384 x 4096 FP32 62 us each, 5.4 TB/s.  Rows
// that do not allow 32-byte accesses go element by element, consecutive over the warp (5003 x 1361 BF16:
// 12 and 10 us).
#include "act.cuh"
#include "kernels.cuh"

namespace gift {

namespace {

constexpr int kActThreads = 256;

template <int F, typename E, bool VEC>
__global__ void __launch_bounds__(kActThreads) k_act_encode(const E *__restrict__ x, int T, int d, int groups,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                            int *status) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (PieceWalk w((size_t)blockIdx.x * (kActThreads / 32) + (threadIdx.x >> 5), (size_t)gridDim.x * (kActThreads / 32),
                   (d + kPiece - 1) / kPiece);
       w.t < T; w.next()) {
    const int c0 = w.p * kPiece, n = d - c0;
    const size_t at = (size_t)w.t * d + c0;
    Raw<E> r;
    load_piece<VEC>(x + at, n, lane, r);
    float2 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r.pair(k);
    bad |= encode_piece<F, VEC>(v, n, lane, codes + at, scales + (size_t)w.t * groups + w.p * 4);
  }
  if (bad) set_status(status, GIFT_ERR_NONFINITE);
}

template <int F, typename E, bool VEC>
__global__ void __launch_bounds__(kActThreads) k_act_decode(const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, int T, int d,
                                                            int groups, E *__restrict__ out, int *status) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (PieceWalk w((size_t)blockIdx.x * (kActThreads / 32) + (threadIdx.x >> 5), (size_t)gridDim.x * (kActThreads / 32),
                   (d + kPiece - 1) / kPiece);
       w.t < T; w.next()) {
    const int c0 = w.p * kPiece, n = d - c0;
    const size_t at = (size_t)w.t * d + c0;
    RawCodes<> r;
    load_codes<VEC>(codes + at, scales + (size_t)w.t * groups + w.p * 4, n, lane, r);
    float2 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = code_pair<F, VEC>(r, k);
    store_piece<VEC>(out + at, n, lane, v);
    // a marked group's first value is NaN whatever its code
    bad |= VEC ? r.s == kActBad
               : (r.s & 0xFFu) == kActBad || ((r.s >> 8) & 0xFFu) == kActBad || ((r.s >> 16) & 0xFFu) == kActBad ||
                     (r.s >> 24) == kActBad;
  }
  if (bad) set_status(status, GIFT_ERR_NONFINITE);
}

// a warp per piece, up to the resident CTAs of the context's SMs
int act_grid(const Launch &L, int T, int d) {
  const size_t pieces = (size_t)T * ((d + kPiece - 1) / kPiece), ctas = (pieces + kActThreads / 32 - 1) / (kActThreads / 32);
  const size_t most = (size_t)L.sms * 8;
  return (int)(ctas < most ? ctas : most);
}

template <int F, typename E>
cudaError_t encode(const Launch &L, const void *x, int T, int d, uint8_t *codes, uint8_t *scales) {
  const int groups = (d + kActGroup - 1) / kActGroup, grid = act_grid(L, T, d);
  const E *p = static_cast<const E *>(x);
  if (rows_vec(d, x, codes)) k_act_encode<F, E, true><<<grid, kActThreads, 0, L.stream>>>(p, T, d, groups, codes, scales, L.status);
  else k_act_encode<F, E, false><<<grid, kActThreads, 0, L.stream>>>(p, T, d, groups, codes, scales, L.status);
  return cudaGetLastError();
}

template <int F, typename E>
cudaError_t decode(const Launch &L, const uint8_t *codes, const uint8_t *scales, int T, int d, void *out) {
  const int groups = (d + kActGroup - 1) / kActGroup, grid = act_grid(L, T, d);
  E *p = static_cast<E *>(out);
  if (rows_vec(d, out, codes)) k_act_decode<F, E, true><<<grid, kActThreads, 0, L.stream>>>(codes, scales, T, d, groups, p, L.status);
  else k_act_decode<F, E, false><<<grid, kActThreads, 0, L.stream>>>(codes, scales, T, d, groups, p, L.status);
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
