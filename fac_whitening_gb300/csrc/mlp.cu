// The feed-forward block's products, host side: operands as the tensor-core kernel reads them (product.cuh), its
// tiles and slices, and the kernels before and after it.
#include <cmath>

#include "operand.cuh"
#include "product.cuh"

namespace gift {

namespace {

using product::Params;

// ---- operands with 16-byte aligned rows, made by one launch -------------------------------------------
// FP32 -> three BF16 terms, or BF16 rows of another pitch; each operand has CTAs of its own.
struct Operands {
  int n;
  struct One {
    const void *src;
    uint8_t *dst;
    int rows, cols, ld;   // ld: elements
    int ctas;
  } op[4];
};

__global__ void __launch_bounds__(256) k_operands(const __grid_constant__ Operands O, bool bf16) {
  grid_release();
  int cta = blockIdx.x;
  for (int i = 0; i < O.n; ++i) {
    const Operands::One &o = O.op[i];
    if (cta < o.ctas) {
      if (bf16)
        repitch(static_cast<const uint8_t *>(o.src), o.rows, (size_t)o.cols * 2, (size_t)o.ld * 2, o.dst, cta, o.ctas);
      else
        bf16_terms(static_cast<const float *>(o.src), o.rows, o.cols, o.ld, reinterpret_cast<uint16_t *>(o.dst), cta,
                   o.ctas);
      return;
    }
    cta -= o.ctas;
  }
}

// ---- sums of slices of k -> the linear product's epilogue ------------------------------------------------
// A thread has eight columns of one row of a tile (one draw of dropout's bits); slices are added in order.
constexpr int kJoinThreads = 128;
template <typename E>
__global__ void __launch_bounds__(kJoinThreads) k_join_linear(const __grid_constant__ Params P, bool vec) {
  const int groups = P.bn / 8, tiles = P.mt * P.nt - P.whole;
  const size_t all = (size_t)tiles * product::kTileRows * groups, plane = (size_t)product::kTileRows * P.bn;
  grid_wait();
  const Draw draw(P.drop);
  const E *residual = static_cast<const E *>(P.in0);
  E *y = static_cast<E *>(P.out0);
  for (size_t i = (size_t)blockIdx.x * kJoinThreads + threadIdx.x; i < all;
       i += (size_t)gridDim.x * kJoinThreads) {
    const int tile = (int)(i / ((size_t)product::kTileRows * groups));
    const int in = (int)(i - (size_t)tile * product::kTileRows * groups);
    const int r = in / groups, g = in - r * groups;
    int m, n;
    product::tile_place(P, P.whole + tile, m, n);
    const int row = m * product::kTileRows + r, col = n * P.bn + 8 * g, left = P.N - col;
    if (row >= P.T || left <= 0) continue;
    const float *p = P.part + (size_t)tile * P.slices * plane + (size_t)r * P.bn + 8 * g;
    float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
#pragma unroll 8
    for (int s = 1; s < P.slices; ++s) {
      const float4 x = *reinterpret_cast<const float4 *>(p + s * plane);
      const float4 z = *reinterpret_cast<const float4 *>(p + s * plane + 4);
      a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
      b = make_float4(b.x + z.x, b.y + z.y, b.z + z.z, b.w + z.w);
    }
    float2 v[4] = {{a.x, a.y}, {a.z, a.w}, {b.x, b.y}, {b.z, b.w}};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (P.bias0) {
        if (2 * k < left) v[k].x += P.bias0[col + 2 * k];
        if (2 * k + 1 < left) v[k].y += P.bias0[col + 2 * k + 1];
      }
    if (draw.below) draw.apply8(v, row, col / 8);
    const size_t at = (size_t)row * P.N + col;
    if (sizeof(E) == 2 && vec) {   // eight columns are 16 bytes
      if (residual) {
        const product::Piece<__nv_bfloat16> r(*reinterpret_cast<const uint4 *>(residual + at));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = add2(v[k], r.v[k]);
      }
      *reinterpret_cast<uint4 *>(y + at) = product::pack_piece<__nv_bfloat16>(v);
      continue;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e >= left) break;
      float x = e & 1 ? v[e / 2].y : v[e / 2].x;
      if (residual) x += ld1(residual + at + e);
      st1(y + at + e, x);
    }
  }
}

// ---- host ---------------------------------------------------------------------------------------------
constexpr int kSegment = 16, kSegment6 = 6;   // most stages of a segment: 1024 k, or one block of 64 k of FP32's terms

struct Source {
  const void *p;
  int rows, cols;
  int box;   // rows of a TMA box
};

// The tensor T x N that an epilogue's buffers are copied to or from: boxes of 32 rows x 128 bytes, or 64 codes.
bool unit_map(CUtensorMap *m, CUtensorMapDataType type, int size, const void *base, int T, int N) {
  const auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)T}, stride = (cuuint64_t)N * size;
  const cuuint32_t box[2] = {size == 1 ? 64u : 128u / size, 32}, one[2] = {1, 1};
  return enc(m, type, 2, const_cast<void *>(base), dims, &stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             size == 1 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An epilogue's tensors by TMA, where all their rows and pointers are 16-byte aligned (the codes' too); null ones are not
// used.  vec: whether they are.
bool unit_maps(product::IoMaps &io, bool bf16, int T, int N, const void *t0, const void *t1, const void *t2,
               const void *t3, const void *codes, bool &vec) {
  const void *t[4] = {t0, t1, t2, t3};
  vec = N % (codes ? 16 : bf16 ? 8 : 4) == 0 && aligned16(codes);
  for (const void *p : t) vec = vec && aligned16(p);
  if (!vec) return true;
  for (int i = 0; i < 4; ++i)
    if (t[i] && !unit_map(&io.m[i], bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                          bf16 ? 2 : 4, t[i], T, N))
      return false;
  return !codes || unit_map(&io.m[3], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, T, N);
}

size_t operand_bytes(bool bf16, int rows, int cols) {
  return ((size_t)rows * pad16((size_t)cols * 2) * (bf16 ? 1 : 3) + 255) / 256 * 256;
}

// The tensor maps of up to four operands; those that TMA cannot read as they lie are made in `ws`, in their
// order, by one launch (`made`).
cudaError_t operands(const Launch &L, bool bf16, const Source *src, int n, uint8_t *ws, CUtensorMap *maps, bool &made) {
  Operands O{};
  int grid = 0;
  for (int i = 0; i < n; ++i) {
    const Source &s = src[i];
    size_t pitch = (size_t)s.cols * 2;
    const void *at = s.p;
    if (!bf16 || pitch % 16 || !aligned16(at)) {
      pitch = pad16(pitch);
      Operands::One &o = O.op[O.n++];
      o.src = s.p;
      o.dst = ws;
      o.rows = s.rows;
      o.cols = s.cols;
      o.ld = (int)(pitch / 2);
      const size_t all = spans(s.rows, s.cols, kSpan), ctas = (all + 7) / 8, most = (size_t)L.sms * 8;
      o.ctas = (int)(ctas < most ? ctas : most);
      grid += o.ctas;
      at = ws;
    }
    ws += operand_bytes(bf16, s.rows, s.cols);
    if (!boxes(&maps[i], true, at, s.rows, s.cols, pitch, bf16 ? 1 : 3, s.box)) return cudaErrorInvalidValue;
  }
  made = grid > 0;
  if (made) k_operands<<<grid, 256, 0, L.stream>>>(O, bf16);
  return cudaGetLastError();
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A launch's tiles: 256 rows x bn columns; the first `whole` are an item each, the others are cut into slices of k.
struct Plan {
  int bn, whole, slices;
  double cost;
};

// Microseconds of a stage, and of a tile's epilogue: what it computes and stores after its last MMA.  A stage of fewer
// columns is bound by its loads: 0.285, 0.25, 0.2 and 0.19 us at 256, 192, 128 and 64 columns (9728 x 4096 x 1536).  An
// epilogue of 256 columns takes 2 us (linear; counted as 2.5, and 1.5 to 3.5 give the same times on 14 of 15 shapes), 5 (gated
// backward) and 4 to 8 with FP32's twice as many bytes; it runs beside the next tile's product, so the last one counts.
struct TileCost {
  bool bf16;
  double epilogue;   // of 256 columns
  double stages(int bn, int blocks) const {
    return blocks * (bf16 ? 1 : 6) * (bn == 256 ? 0.285 : bn == 192 ? 0.25 : bn == 128 ? 0.2 : 0.19) + 0.5;
  }
  double end(int bn) const { return epilogue * (bf16 ? 1.0 : 1.6) * bn / 256; }
  double waves(int n, int bn, int blocks) const {
    const double a = stages(bn, blocks), b = end(bn);
    return n * (a > b ? a : b);
  }
};
constexpr double kLinearEnd = 2.5, kGatedEnd = 5.0;

// The width with the least time.  With `cut`, the tiles after the last full wave of pairs are cut into slices of k where
// that wave and the kernel that joins the slices (its launch and 6 TB/s) end sooner than a wave of whole tiles would:
// 16384 x 6144 x 1536 has 384 tiles of 256 on 76 pairs, 195 us with six waves, 182 with five and slices; 16384 x 12288 x 1536
// 368 and 334.
Plan plan_of(int sms, const TileCost &c, int T, int N, int kb, bool cut) {
  const int pairs = sms / 2 > 1 ? sms / 2 : 1;
  const int mt = ceil_div(T, product::kTileRows);
  Plan best{256, 0, 1, 1e300};
  for (int bn = 256; bn >= 64; bn -= 64) {
    const int tiles = mt * ceil_div(N, bn), full = tiles / pairs, rest = tiles - full * pairs;
    const double whole = c.waves(full + (rest > 0), bn, kb) + c.end(bn);
    if (whole < best.cost) best = Plan{bn, tiles, 1, whole};
    for (int s = 2; cut && s <= 32 && s <= kb && rest; ++s) {
      const double cost = c.waves(full, bn, kb) + c.waves(ceil_div(rest * s, pairs), bn, ceil_div(kb, s)) + c.end(bn) +
                          3.0 + 2.0 * rest * s * (T < product::kTileRows ? T : product::kTileRows) * bn * 4 / 6.0e6;
      if (cost < best.cost) best = Plan{bn, tiles - rest, s, cost};
    }
  }
  return best;
}
Plan plan_linear(int sms, bool bf16, int T, int N, int kb) {
  return plan_of(sms, TileCost{bf16, kLinearEnd}, T, N, kb, true);
}

int pairs_of(const Launch &L) { return L.sms / 2 > 1 ? L.sms / 2 : 1; }

Params params_of(const Launch &L, bool bf16, int T, int N, int columns, int bn, bool b_mn, int kb) {
  Params P{};
  P.T = T;
  P.N = N;
  P.mt = ceil_div(T, product::kTileRows);
  P.nt = ceil_div(N, columns);
  P.group = 8;
  P.slices = 1;
  P.whole = P.items = P.mt * P.nt;
  P.kb = P.kb1 = kb;
  // segments of equal length, so that none ends long before the next is folded
  P.head = P.seg = bf16 ? ceil_div(kb, ceil_div(kb, kSegment)) : kSegment6;
  P.bn = bn;
  P.idesc = tc::idesc_bf16(256, bn) | (b_mn ? 1u << 16 : 0u);
  P.budget = L.barrier_wait;
  return P;
}

// Stages of the segments of a BF16 product whose results are also kept in 8 bits: of the first two, which the epilogue needs
// long, and of the others.  Error of the values that the codes stand for, and changed codes, over those of a plain FP32
// product, and the product's time, 16384 tokens x 6144 (32768 x 16384 at 4096 k); right, longer ones of 0.61 sqrt(k / 64)
// stages, at least 3, the first two twice as long:
//      k   stages  error  codes      us     error  codes     us
//    256     2, 2   1.10   1.11   162.5      1.19   1.45   162.5
//    512     2, 2   1.14   0.87     253      1.33   1.12     237
//    768     2, 2   1.09   0.75     300      1.88   1.82     226
//   1024     3, 2   0.88   0.77     328      1.46   1.52     289
//   1536     4, 2   0.97   0.70     410      1.23   1.08     381
//   2048     5, 2   0.89   0.71     498      0.99   0.86     484
//   4096     8, 3   0.80   0.67    4710      1.00   0.90    4570
// Truncation moves a sum towards zero, the large ones most, in proportion to a segment's length; a plain sum's roundings
// grow with the square root of k.  One stage a segment: 0.94 at 256 k, but 39 % more time.
void checkpoint_segments(int kb, int &head, int &seg) {
  const int root = (int)(std::sqrt((double)kb) + 0.5), line = 1 + kb / 8;
  head = line < root ? line : root;
  if (head < 2) head = 2;
  if (head > kSegment) head = kSegment;
  seg = (head + 1) / 3 > 2 ? (head + 1) / 3 : 2;
}

}  // namespace

MlpWs gated_forward_layout(bool bf16, int T, int f, int d) {
  MlpWs w;
  w.operand_bytes = operand_bytes(bf16, T, d) + 2 * operand_bytes(bf16, f, d);
  return w;
}

cudaError_t launch_gated_forward(const Launch &L, bool bf16, const GatedForward &a) {
  CUtensorMap maps[4];
  const Source src[3] = {{a.x, a.T, a.d, 128}, {a.Wg, a.f, a.d, 128}, {a.Wu, a.f, a.d, 128}};
  CUtensorMap made_maps[3];
  bool made;
  const cudaError_t e = operands(L, bf16, src, 3, a.ws, made_maps, made);
  if (e != cudaSuccess) return e;
  maps[0] = maps[1] = made_maps[0];
  maps[2] = made_maps[1];
  maps[3] = made_maps[2];
  Params P = params_of(L, bf16, a.T, a.f, 128, 256, false, ceil_div(a.d, product::kK));
  if (bf16 && a.codes) checkpoint_segments(P.kb, P.head, P.seg);
  P.group = 16;
  P.fn = a.fn;
  P.fmt = a.fmt;
  P.groups = ceil_div(a.f, kActGroup);
  P.bias0 = a.bg;
  P.bias1 = a.bu;
  P.out0 = a.h;
  P.out1 = a.gate;
  P.out2 = a.up;
  P.codes = a.codes;
  P.scales = a.scales;
  product::IoMaps io{};
  bool vec;
  if (!unit_maps(io, bf16, a.T, a.f, a.h, a.gate, a.up, nullptr, a.codes, vec)) return cudaErrorInvalidValue;
  return product::launch_gated_forward(L, bf16, vec, P, maps, io, pairs_of(L), made);
}

MlpWs gated_backward_layout(bool bf16, int T, int d_out, int f) {
  MlpWs w;
  w.operand_bytes = operand_bytes(bf16, T, d_out) + operand_bytes(bf16, d_out, f);
  return w;
}

cudaError_t launch_gated_backward(const Launch &L, bool bf16, const GatedBackward &a) {
  const Source src[2] = {{a.dy, a.T, a.d_out, 128}, {a.W, a.d_out, a.f, 64}};
  CUtensorMap made_maps[2];
  bool made;
  const cudaError_t e = operands(L, bf16, src, 2, a.ws, made_maps, made);
  if (e != cudaSuccess) return e;
  const CUtensorMap maps[4] = {made_maps[0], made_maps[0], made_maps[1], made_maps[1]};
  const int kb = ceil_div(a.d_out, product::kK);
  const int bn = plan_of(L.sms, TileCost{bf16, kGatedEnd}, a.T, a.f, kb, false).bn;
  Params P = params_of(L, bf16, a.T, a.f, bn, bn, true, kb);
  P.fn = a.fn;
  P.in0 = a.gate;
  P.in1 = a.up;
  P.out0 = a.dgate;
  P.out1 = a.dup;
  product::IoMaps io{};
  bool vec;
  if (!unit_maps(io, bf16, a.T, a.f, a.gate, a.up, a.dgate, a.dup, nullptr, vec)) return cudaErrorInvalidValue;
  return product::launch_gated_backward(L, bf16, vec, P, maps, io, pairs_of(L), made);
}

namespace {

// A product with the linear epilogue, its last tiles in slices.
cudaError_t linear(const Launch &L, bool bf16, bool mn, const Plan &p, Params P, const CUtensorMap *maps, bool made,
                   float *part) {
  P.whole = p.whole;
  P.slices = p.slices;
  const int cut = P.mt * P.nt - p.whole;
  P.items = p.whole + cut * p.slices;
  P.part = part;
  product::IoMaps io{};
  bool vec;
  if (!unit_maps(io, bf16, P.T, P.N, P.in0, nullptr, P.out0, nullptr, nullptr, vec)) return cudaErrorInvalidValue;
  const cudaError_t e = product::launch_linear(L, bf16, vec, mn, P, maps, io, pairs_of(L), made);
  if (e != cudaSuccess || !cut) return e;
  const size_t ctas = (size_t)cut * product::kTileRows * (P.bn / 8) / kJoinThreads, most = (size_t)L.sms * 16;
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  return bf16 ? launch_after(L.stream, k_join_linear<__nv_bfloat16>, grid, kJoinThreads, P, vec)
              : launch_after(L.stream, k_join_linear<float>, grid, kJoinThreads, P, vec);
}

size_t part_floats(const Plan &p, int T, int N) {
  const size_t tiles = (size_t)ceil_div(T, product::kTileRows) * ceil_div(N, p.bn);
  return (tiles - p.whole) * p.slices * product::kTileRows * p.bn;
}

}  // namespace

MlpWs linear_forward_layout(int sms, bool bf16, int T, int d_out, int d_in) {
  MlpWs w;
  w.operand_bytes = operand_bytes(bf16, T, d_in) + operand_bytes(bf16, d_out, d_in);
  w.part_floats = part_floats(plan_linear(sms, bf16, T, d_out, ceil_div(d_in, product::kK)), T, d_out);
  return w;
}

cudaError_t launch_linear_forward(const Launch &L, bool bf16, const LinearForward &a) {
  const int kb = ceil_div(a.d_in, product::kK);
  const Plan p = plan_linear(L.sms, bf16, a.T, a.d_out, kb);
  const Source src[2] = {{a.x, a.T, a.d_in, 128}, {a.W, a.d_out, a.d_in, p.bn / 2}};
  CUtensorMap made_maps[2];
  bool made;
  const cudaError_t e = operands(L, bf16, src, 2, a.ws, made_maps, made);
  if (e != cudaSuccess) return e;
  const CUtensorMap maps[4] = {made_maps[0], made_maps[0], made_maps[1], made_maps[1]};
  Params P = params_of(L, bf16, a.T, a.d_out, p.bn, p.bn, false, kb);
  P.bias0 = a.bias;
  P.in0 = a.residual;
  P.out0 = a.y;
  P.drop.rng = a.rng;
  P.drop.below = a.below;
  P.drop.site = a.site;
  P.drop.scale = 65536.0f / (float)(65536 - a.below);
  return linear(L, bf16, false, p, P, maps, made, a.part);
}

MlpWs input_grad_layout(int sms, bool bf16, int T, int d_out, int d_in) {
  MlpWs w;
  w.operand_bytes = 2 * (operand_bytes(bf16, T, d_out) + operand_bytes(bf16, d_out, d_in));
  const int kb = ceil_div(d_out, product::kK);   // one pair of operands, or two
  const size_t one = part_floats(plan_linear(sms, bf16, T, d_in, kb), T, d_in),
               two = part_floats(plan_linear(sms, bf16, T, d_in, 2 * kb), T, d_in);
  w.part_floats = one > two ? one : two;
  return w;
}

cudaError_t launch_input_grad(const Launch &L, bool bf16, const InputGrad &a) {
  const int kb = ceil_div(a.d_out, product::kK), n = a.delta2 ? 2 : 1;
  const Plan p = plan_linear(L.sms, bf16, a.T, a.d_in, n * kb);
  const Source src[4] = {{a.delta, a.T, a.d_out, 128},
                         {a.W, a.d_out, a.d_in, 64},
                         {a.delta2, a.T, a.d_out, 128},
                         {a.W2, a.d_out, a.d_in, 64}};
  CUtensorMap m[4];
  bool made;
  const cudaError_t e = operands(L, bf16, src, 2 * n, a.ws, m, made);
  if (e != cudaSuccess) return e;
  const CUtensorMap maps[4] = {m[0], m[n == 2 ? 2 : 0], m[1], m[n == 2 ? 3 : 1]};
  Params P = params_of(L, bf16, a.T, a.d_in, p.bn, p.bn, true, n * kb);
  P.kb1 = kb;
  P.out0 = a.dx;
  return linear(L, bf16, true, p, P, maps, made, a.part);
}

}  // namespace gift
