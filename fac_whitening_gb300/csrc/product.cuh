// The feed-forward block's products on the 5th-generation tensor cores: one persistent kernel, its epilogue by
// operator.  out[t][n] = sum_k A[t][k] B[k][n], A the T tokens' rows (K contiguous), B a weight matrix read as it
// lies in memory, K-major (n x k: a forward product) or MN-major (k x n: a product with its transpose).
//
// A pair of CTAs (a cluster of two SMs, cta_group::2) owns 256 tokens x up to 256 columns: each CTA holds 128 of
// the tokens and half of B's columns.  Per CTA:
//   warps 0, 2   TMA: stages of 64 k, A's 128 x 64 and B's up to 128 x 64 elements;
//   warp 1       the pair's first CTA issues 256 x N x 16 MMAs (both CTAs' copies complete on its barriers);
//   warps 4-11   fold and epilogue: a thread has one token and half of the tile's columns.
// The tensor core truncates its sums, so a segment of at most 1024 k goes into one of two accumulators in tensor memory
// and is added to FP32 registers to nearest while the other is filled.  The epilogue runs from those registers while
// the next tile's first two segments are multiplied: 1536 k are two segments, and the epilogue has a tile's whole time.
// An 8-bit checkpoint of h tells FP32's last bits (the codes of values next to a border), so a forward product that
// makes one has shorter segments (checkpoint_segments): 128 k of 512, 256 of 1536, 512 of 4096 in the first two, which
// the epilogue needs, fewer in the others.
// The gated forward product takes its two projections as one product of 128 + 128 columns: the first CTA loads
// the gate's rows, the second the other projection's, and both halves of a row meet in one thread.
// FP32 operands are three BF16 terms each (operand.cuh); a block of 64 k then takes six stages, the products i + j <= 2
// of terms i and j; what is dropped is below 2^-23 of |A_k B_k|.  A block is a segment and the small products come
// first, so that only the last stage's four steps truncate at the sum's size: outputs are 0.9e-7 off at 256 k, 1.1e-7 at
// 1021 and 4096 (relative Frobenius; a plain FP32 product 2.9e-7, 5.7e-7 and 1.1e-6; segments of two blocks 6e-7).
// What bounds it.  A stage's MMAs of 256 columns take 512 clocks, its 32 KB cross from L2 at up to 64 bytes a clock: 540 to
// 560 clocks a stage.  16384 x 12288 x 1536 input gradient 330 us, 1.87 PFLOP/s; 16384 x 6144 x 1536 linear with dropout
// and residual 180 us; 16384 x 1536 x 6144 gated forward 414 us with the checkpoint, 345 without, backward 232 us (g, u and
// their gradients are 805 MB: 157 us without them); 32768 x 4096 x 16384 gated forward with it 4.6 to 5.3 ms.  A
// library's BF16 product by itself takes 335, 171, 308 (both projections in one), 156 us and, where that took 5.3 ms, 4.7.  Small ones: a start of
// 1 us, 1 us to the first stage, 3 us for a BF16 epilogue.
// Every mbarrier wait is bounded by the context's GIFT_OPT_BARRIER_WAIT and reports GIFT_ERR_TIMEOUT; a warp
// leaves as one, and the copies and MMAs in flight are waited for before the CTA leaves.
#pragma once

#include <type_traits>

#include "act.cuh"
#include "dropout.cuh"
#include "gate.cuh"
#include "kernels.cuh"
#include "operand.cuh"
#include "pair.cuh"

namespace gift {

namespace product {

constexpr int kK = 64;                      // k of a stage
constexpr int kABytes = 128 * kK * 2;       // a CTA's rows of A in a stage, and its most columns of B
constexpr int kStage = 2 * kABytes;
constexpr int kBox = kK * 128;              // bytes of an MN-major box: 64 columns
constexpr int kThreads = 384;
constexpr int kEpiWarp = 4, kEpiWarps = 8;
constexpr int kTileRows = 256;
constexpr int kUnit = 32 * 128;             // bytes of an epilogue buffer: 32 rows of 64 BF16 or 32 FP32 columns

enum Op { GATED_FORWARD, GATED_BACKWARD, LINEAR };

// Shared memory: a ring of stages, and epilogue buffers for each of its warps (forward: used in turn, so that a store is
// read while the next buffer is written, 2 % of 16384 x 1536 x 6144 although a stage had to go; backward: the
// gate's and the other projection's unit side by side, the gradients in their place).
template <int OP>
struct Cfg {
  static constexpr int stages = OP == LINEAR ? 6 : 5;
  static constexpr int bufs = OP == LINEAR ? 1 : 2;
  static constexpr int smem = stages * kStage + kEpiWarps * bufs * kUnit + 1024;
};
struct IoMaps {
  CUtensorMap m[4];   // boxes of 32 rows x 128 bytes: in0, in1, out0, out1; forward: out0 to out2 and the codes (64 bytes)
};

struct Params {
  int T, N;               // rows and columns of the output
  int mt, nt, group;      // tiles, and rows of tiles that are taken together
  int whole, slices;      // the first `whole` tiles are an item each, the others (linear only) `slices` each
  int items;
  int kb, kb1;            // blocks of 64 k, and those of the first pair of operands
  int head, seg;          // stages of an item's first two segments, and of the others
  int bn;                 // columns of a tile, a multiple of 64
  uint32_t idesc;
  long long budget;       // clocks of a wait
  // epilogue
  int fn, fmt, groups;
  const float *bias0, *bias1;   // nullable
  const void *in0, *in1;        // gated backward: gate, up; linear: in0 the residual (nullable)
  void *out0, *out1, *out2;     // forward: h, gate, up (nullable both); backward: dgate, dup; linear: y
  uint8_t *codes, *scales;      // nullable: h's 8-bit checkpoint
  Dropout drop;
  float *part;                  // slices: [tile - whole][slice][256][bn]
};

// Row m and column n of tiles of a tile.  Tiles are in groups of rows of tiles, column by column within a group: the
// pairs that run at the same time share both operands in L2.  Groups of 2, 4, 8, 16 and 32 rows: 16384 x 1536 x 6144 gated
// forward 365, 367, 353, 345, 355 us, 32768 x 4096 x 16384 with the checkpoint 5510, 5340, 5330, 5280, 5380 (16 there);
// 16384 x 6144 x 1536 linear 181, 183, 183, 187, 197, 32768 x 4096 x 16384 gated backward 2950, 2840, 2800, 2800, 2840 (8).
__host__ __device__ inline void tile_place(const Params &P, int tile, int &m, int &n) {
  const int per = P.group * P.nt, g = tile / per, rem = tile - g * per;
  const int rows = P.mt - P.group * g < P.group ? P.mt - P.group * g : P.group;
  n = rem / rows;
  m = P.group * g + rem - n * rows;
}

struct Item {
  int m, n, slice, k0, k1;   // tile, its slice (-1: all of it), blocks of 64 k
  __device__ __forceinline__ Item(const Params &P, int item) {
    int tile = item;
    slice = -1;
    k0 = 0;
    k1 = P.kb;
    if (item >= P.whole) {
      const int cut = P.mt * P.nt - P.whole, i = item - P.whole;
      slice = i / cut;
      tile = P.whole + i - slice * cut;
      k0 = (int)((long long)P.kb * slice / P.slices);
      k1 = (int)((long long)P.kb * (slice + 1) / P.slices);
    }
    tile_place(P, tile, m, n);
    at = tile - P.whole;
  }
  int at;   // the tile's place among the cut ones
};

constexpr int kMostStages = 6;
struct __align__(16) Shared {
  uint64_t full[kMostStages], empty[kMostStages];   // first CTA: loaded in both; multiplied (in both CTAs)
  uint64_t in[kEpiWarps];                           // an epilogue warp's buffer: loaded
  uint64_t dfull[2], dempty[2];             // accumulators: summed; folded by both CTAs
  uint64_t met[4];                          // a row's two column halves have left their scale bytes
  uint64_t drained;
  uint8_t scale[2][2][128];                 // [tile parity][half][row]: the scale byte that the half's columns ask for
  uint32_t issued[4];                       // copies that the pair's TMA threads made, and whether one gave up
  uint32_t tmem;
  volatile int failed;
};
constexpr uint32_t kGaveUp = 1u << 31;

// D (+)= A[smem] B[smem], one 256 x N x 16 step over both CTAs
__device__ __forceinline__ void mma_pair_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            uint32_t accumulate) {
  // 128-byte swizzle, 8-row (or 8-k) groups 1024 bytes apart
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
      "mov.b64 ad, {%1, %5};\n\t"
      "mov.b64 bd, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %3, p;\n\t}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(hi)
      : "memory");
}

// Barriers and copies by shared-memory address
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool test_wait_at(uint32_t bar, uint32_t parity) {   // looks, does not wait
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void expect_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// Of shared memory of the pair's CTA r: its address, an arrival with `bytes` to come, a word's write; and a copy into this
// CTA that completes on a barrier of either.  A copy that the first CTA has to be told of by the second costs a
// stage of latency: 16384 x 1536 x 6144 gated forward 378 us with a thread that passed them on, 365 without.
__device__ __forceinline__ uint32_t of_cta(uint32_t at, uint32_t r) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(at), "r"(r));
  return a;
}
__device__ __forceinline__ void expect_in_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void write_in_cluster(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void load_in_cluster(uint32_t dst, const CUtensorMap *tmap, int x, int y, int z,
                                                uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// The next slot of a ring of N, and the parity of its uses
template <int N>
__device__ __forceinline__ void advance(uint32_t &at, uint32_t &parity) {
  if (++at == N) {
    at = 0;
    parity ^= 1u;
  }
}

// ---- units: a lane's 128 bytes of one row, of 32 consecutive rows per warp ------------------------------
// A warp's buffer holds them in the 128-byte swizzle of its tensor map: 16-byte piece j of row r at j ^ (r % 8), so that
// eight lanes' pieces do not meet in a bank.  TMA moves whole buffers: a lane's own accesses to 32 rows cost the load
// and store unit 67 clocks for each 32 bytes a lane (the stores of g and u 4300 clocks a tile, of 12300).
__device__ __forceinline__ uint32_t piece_at(uint32_t buf, int lane, int j) {
  return buf + lane * 128 + ((j ^ (lane & 7)) << 4);
}
__device__ __forceinline__ uint4 read_piece(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void write_piece(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// A piece's columns (8 BF16 or 4 FP32) as pairs
template <typename E>
struct Piece {
  static constexpr int pairs = sizeof(E) == 2 ? 4 : 2;
  float2 v[pairs];
  Piece() = default;
  __device__ __forceinline__ explicit Piece(uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < pairs; ++k)
      v[k] = sizeof(E) == 2 ? make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u))
                            : make_float2(__uint_as_float(w[2 * k % 4]), __uint_as_float(w[(2 * k + 1) % 4]));
  }
};
template <typename E>
__device__ __forceinline__ uint4 pack_piece(const float2 *v) {
  if (sizeof(E) == 2)
    return make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y),
                      pack_bf16(v[3].x, v[3].y));
  return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
}
// Copies between a buffer and its place in a tensor; stores of a thread are waited for in groups.
__device__ __forceinline__ void load_unit(uint32_t buf, const CUtensorMap *map, int col, int row, uint32_t bar) {
  expect_at(bar, kUnit);
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          buf),
      "l"(map), "r"(col), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void store_unit(uint32_t buf, const CUtensorMap *map, int col, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n"
      "cp.async.bulk.commit_group;\n" ::"l"(map),
      "r"(col), "r"(row), "r"(buf)
      : "memory");
}
// A unit by the warp's own copies (8 lanes to a row, 32 rows), for the gated backward product: TMA's queue serves the
// product's operands there while these come from HBM (16384 x 1536 x 6144: 271 us by TMA, 248 so).
template <typename E>
__device__ __forceinline__ void load_rows(uint32_t buf, const void *base, size_t ld, int row0, int rows, int col, int n) {
  const int lane = threadIdx.x & 31, j = lane & 7;
  constexpr int per = 16 / sizeof(E);
  const E *p = static_cast<const E *>(base) + (size_t)row0 * ld + col + per * j;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    if (r < rows && per * j < n)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(piece_at(buf, r, j)), "l"(p + (size_t)r * ld)
                   : "memory");
  }
}
__device__ __forceinline__ void loads_done() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }
// a thread's stores have been read, but for the last N
template <int N = 0>
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }

// ---- units of rows of any alignment, 8 lanes to a row ------------------------------------------------------
// Rows start anywhere in a 16-byte block.  A load takes the two aligned blocks that a piece lies in and shifts; a store
// writes the aligned blocks that the unit's part of a row covers, and the elements before and after them one by one
// (5003 x 1361 x 2731 gated backward, every access an element wide: 200 us).
template <typename E>
__device__ __forceinline__ void load_any(uint32_t buf, const void *base, int T, int N, int row0, int rows, int col) {
  const int lane = threadIdx.x & 31, j = lane & 7;
  const uintptr_t lo = (uintptr_t)base, hi = lo + (size_t)T * N * sizeof(E);
  const size_t step = (size_t)4 * N * sizeof(E);
  uintptr_t at = lo + ((size_t)(row0 + (lane >> 3)) * N + col) * sizeof(E) + 16 * j;
  const uintptr_t from = lo + ((size_t)row0 * N + col) * sizeof(E);
  if (rows >= 32 && from >= lo + 16 && from + 31 * (step / 4) + 160 <= hi) {   // every block is whole
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 a[4], b[4];   // 16 rows' loads before the first store
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uintptr_t p = at + u * step, block = p & ~(uintptr_t)15;
        a[u] = *reinterpret_cast<const uint4 *>(block);
        b[u] = *reinterpret_cast<const uint4 *>(block + (p != block ? 16 : 0));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        write_piece(piece_at(buf, 16 * h + 4 * u + (lane >> 3), j), shifted(a[u], b[u], (int)((at + u * step) & 15)));
      at += 4 * step;
    }
    return;
  }
#pragma unroll 1
  for (int r = lane >> 3; r < 32; r += 4, at += step) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && at < hi) {   // past the row's end: what lies there, never stored
      const int off = (int)(at & 15);
      v = aligned_block(at - off, lo, hi);
      if (off) v = shifted(v, aligned_block(at - off + 16, lo, hi), off);
    }
    write_piece(piece_at(buf, r, j), v);
  }
}
// E's bytes of a buffer's row from byte `from`
template <typename E>
__device__ __forceinline__ void store_element(E *p, uint32_t buf, int r, int from) {
  const uint32_t at = piece_at(buf, r, from >> 4) + (from & 15);
  if constexpr (sizeof(E) == 1) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    *p = (E)v;
  } else if constexpr (sizeof(E) == 2) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    *reinterpret_cast<uint16_t *>(p) = v;
  } else {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    *reinterpret_cast<uint32_t *>(p) = v;
  }
}
// COLS columns of the unit, n of them in the matrix
template <typename E, int COLS>
__device__ __forceinline__ void store_any(uint32_t buf, void *base, int N, int row0, int rows, int col, int n) {
  constexpr int size = sizeof(E);
  const int lane = threadIdx.x & 31, j = lane & 7, len = min(n, COLS) * size;
  E *p = static_cast<E *>(base) + (size_t)(row0 + (lane >> 3)) * N + col;
  constexpr int kRest = (2 * (16 / size - 1) + 7) / 8;   // elements before and after the blocks, by lane
#pragma unroll 4
  for (int r = lane >> 3; r < min(rows, 32); r += 4, p += (size_t)4 * N) {
    const int head = min(len, (int)((0 - (uintptr_t)p) & 15)), blocks = (len - head) >> 4;
    if (j < blocks)
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p) + head + 16 * j) =
          shifted(read_piece(piece_at(buf, r, j)), read_piece(piece_at(buf, r, head ? j + 1 : j)), head);
    const int rest = (len - 16 * blocks) / size, before = head / size;
#pragma unroll
    for (int u = 0; u < kRest; ++u) {
      const int i = j + 8 * u, c = i < before ? i : i + 16 * blocks / size;
      if (i < rest) store_element(p + c, buf, r, c * size);
    }
  }
}

// 16 columns of a lane's own row, rows of a multiple of 16 FP32 in 32-byte aligned buffers
__device__ __forceinline__ void store_own(float *p, const float2 *v) {
  uint32_t r[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    r[2 * k] = __float_as_uint(v[k].x);
    r[2 * k + 1] = __float_as_uint(v[k].y);
  }
  st256(p, r);
  st256(p + 8, r + 8);
}

// 16 codes
template <int F>
__device__ __forceinline__ uint4 pack_codes(const float2 *v, float inv) {
  const float2 s = both(inv);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = mul2(v[2 * k], s), b = mul2(v[2 * k + 1], s);
    w[k] = pack4_fp8<F>(a.x, a.y, b.x, b.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The bias of a warp's up to 32 J columns, n of them in the matrix, a column of each 32 per lane: loaded while the tile is
// multiplied, handed round by shuffles in straight code (loads beside their use, by alignment, took 4300 clocks of a
// small product's only epilogue, most of them for the instructions).
template <int J>
struct Bias {
  float v[J];
  __device__ __forceinline__ void load(const float *bias, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = bias && 32 * j + lane < n ? bias[32 * j + lane] : 0.0f;
  }
  // to 16 columns, the i-th such group
  __device__ __forceinline__ void add(float2 *to, int i) const {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      to[k] = add2(to[k], make_float2(__shfl_sync(0xFFFFFFFFu, v[i / 2], (16 * i + 2 * k) % 32),
                                      __shfl_sync(0xFFFFFFFFu, v[i / 2], (16 * i + 2 * k + 1) % 32)));
  }
};

// acc[0..3] the gate's 64 columns, acc[4..7] the other projection's: a(g) u in their place
template <int FN, bool ACCURATE>
__device__ __forceinline__ void gate_forward(float2 (&acc)[8][8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 g = acc[i][k];
      acc[i][k] = mul2(make_float2(gate_value<FN, ACCURATE>(g.x), gate_value<FN, ACCURATE>(g.y)), acc[4 + i][k]);
    }
}
// dh in `d`: the gate's gradient in its place, the other projection's in `du`; N pairs of columns
template <int FN, bool ACCURATE, int N>
__device__ __forceinline__ void gate_backward(float2 *d, float2 *du, const float2 *g, const float2 *u) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float2 slope, a;
    a.x = gate_slope<FN, ACCURATE>(g[k].x, slope.x);
    a.y = gate_slope<FN, ACCURATE>(g[k].y, slope.y);
    du[k] = mul2(d[k], a);
    d[k] = mul2(mul2(d[k], u[k]), slope);
  }
}
// dropped to 0, or scaled
__device__ __forceinline__ void drop16(const Draw &draw, float2 *v, uint32_t keep) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k].x = keep >> (2 * k) & 1u ? v[k].x * draw.scale : 0.0f;
    v[k].y = keep >> (2 * k + 1) & 1u ? v[k].y * draw.scale : 0.0f;
  }
}

// MN: B is MN-major.
template <int OP, typename E, bool VEC, bool MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_product(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap tm_a0,
              const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b0,
              const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ IoMaps io, int *status) {
  constexpr int kStages = Cfg<OP>::stages, kBufs = Cfg<OP>::bufs;
  static_assert(Cfg<OP>::smem + sizeof(Shared) <= 227 * 1024, "a CTA's shared memory");
  constexpr bool kGated = OP == GATED_FORWARD;
  constexpr bool kAccurate = sizeof(E) == 4;
  constexpr int kTerms = sizeof(E) == 4 ? 6 : 1;
  extern __shared__ uint8_t dsm[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(((uintptr_t)dsm + 1023) & ~(uintptr_t)1023);
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (OP == LINEAR && P.slices > 1) grid_release();   // the kernel that joins the slices

  if (warp == 0) alloc_pair(&sh.tmem);
  if (tid == 96) {   // the maps on their way while the rest is set up
    tc::prefetch_tensormap(&tm_a0);
    tc::prefetch_tensormap(rank && kGated ? &tm_b1 : &tm_b0);
  }
  if (tid == 32) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&sh.full[s], 4);
      tc::mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&sh.dfull[b], 1);
      tc::mbar_init(&sh.dempty[b], 2 * kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) tc::mbar_init(&sh.met[q], 2);
    for (int e = 0; e < kEpiWarps; ++e) tc::mbar_init(&sh.in[e], 1);
    tc::mbar_init(&sh.drained, 1);
    tc::fence_mbar_init();
    sh.failed = 0;
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  // Called by whole warps: the lanes go on together, or none does.  Not patient: gives up where a phase is not over when it is
  // looked at.
  auto hold = [&](uint32_t bar, uint32_t parity, bool patient) {
    if (patient && __all_sync(0xFFFFFFFFu, try_wait_at(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xFFFFFFFFu, patient ? try_wait_at(bar, parity) : test_wait_at(bar, parity))) {
      if (__any_sync(0xFFFFFFFFu, sh.failed || clock64() - t0 > P.budget)) {
        sh.failed = 1;
        set_status(status, GIFT_ERR_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  auto wait = [&](uint64_t *bar, uint32_t parity) { return hold(tc::smem_u32(bar), parity, true); };

  // registers: 168 per thread at launch (504 over the three groups of four warps), redistributed as 2 x 208 + 88
  if (warp < kEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    // Each of these warps walks its loop whole and converged, so that what TMA and the MMAs take stays in uniform
    // registers; one elected thread issues.  A stage's 512 clocks are few for what a warp does between two of them: the
    // loops keep their addresses running, and A and B have a warp each (one for both, its slot and terms computed
    // per stage, took 550 clocks a stage).
    const bool one = elect_one(), patient = P.budget > 0;
    const uint32_t full = of_cta(tc::smem_u32(sh.full), 0), empty = tc::smem_u32(sh.empty);
    const uint32_t ring = tc::smem_u32(sm);
    if (warp == 0 || warp == 2) {
      // ---------------- TMA ----------------
      const bool is_a = warp == 0;
      const int half = P.bn / 2, boxes = half > 64 ? 2 : 1;
      const uint32_t bytes = is_a ? kABytes : MN ? boxes * kBox : half * 128;
      const uint32_t base = ring + (is_a ? 0 : kABytes);
      uint32_t at = 0, parity = 1, g = 0;
      bool ok = true;
      grid_wait();   // the operands that the launch before this one made
      auto stage = [&](const CUtensorMap *map, int k, int y, int term) {
        const uint32_t bar = full + 8 * at, dst = base + at * kStage;
        if (!(ok = hold(empty + 8 * at, parity, patient))) return;
        if (one) {
          expect_in_cluster(bar, bytes);
          if (MN && !is_a) {
            load_in_cluster(dst, map, y, k, term, bar);
            if (boxes == 2) load_in_cluster(dst + kBox, map, y + 64, k, term, bar);
          } else {
            load_in_cluster(dst, map, k, y, term, bar);
          }
        }
        __syncwarp();
        advance<kStages>(at, parity);
        ++g;
      };
      for (int it = pair; it < P.items && ok; it += pairs) {
        const Item w(P, it);
        const int y = is_a ? w.m * kTileRows + 128 * rank : kGated ? 128 * w.n : w.n * P.bn + half * rank;
        auto walk = [&](const CUtensorMap *map, int k, int end) {
          for (; k < end && ok; k += kK) {
            if constexpr (kTerms == 1) {
              stage(map, k, y, 0);
            } else {   // terms (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
              const int t[6] = {is_a ? 2 : 0, 1, is_a ? 0 : 2, is_a ? 1 : 0, is_a ? 0 : 1, 0};
#pragma unroll
              for (int p = 0; p < 6; ++p)
                if (ok) stage(map, k, y, t[p]);
            }
          }
        };
        if (kGated) {
          walk(is_a ? &tm_a0 : rank ? &tm_b1 : &tm_b0, w.k0 * kK, w.k1 * kK);
        } else {
          walk(is_a ? &tm_a0 : &tm_b0, w.k0 * kK, min(w.k1, P.kb1) * kK);
          walk(is_a ? &tm_a1 : &tm_b1, max(w.k0 - P.kb1, 0) * kK, (w.k1 - P.kb1) * kK);
        }
      }
      // The last stages' MMAs are done (and leave no arrival of their commits behind): all copies have landed.
      for (uint32_t r = 1; ok && r <= kStages && r <= g; ++r) {
        const Slot<kStages> s(g - r);
        ok = hold(empty + 8 * s.at, s.parity, patient);
      }
      // the pair's first CTA may have a wait of its own to end before its last commit
      tc::mbar_wait_bounded(&sh.drained, 0, P.budget + kDrain);
      __syncwarp();
      const uint32_t at_issued = tc::smem_u32(&sh.issued[2 * rank + (is_a ? 0 : 1)]);
      if (one)
        for (uint32_t r = 0; r < 2; ++r) write_in_cluster(of_cta(at_issued, r), g | (ok ? 0u : kGaveUp));
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA ----------------
      const uint32_t b_lead = MN ? (uint32_t)(kBox >> 4) << 16 : 1u << 16, b_step = MN ? 128u : 2u;
      const uint32_t loaded = tc::smem_u32(sh.full), dempty = tc::smem_u32(sh.dempty), idesc = P.idesc;
      const int head = P.head, seg = P.seg;
      uint32_t at = 0, parity = 0, n = 0;   // slot, segments
      bool ok = true, there = false;        // there: the stage was seen to be loaded
      grid_wait();   // no wait's budget is spent on the launch that makes the operands
      for (int it = pair; it < P.items && ok; it += pairs) {
        const Item w(P, it);
        for (int left = (w.k1 - w.k0) * kTerms, i = 0, len; left > 0 && ok; left -= len, ++i, ++n) {
          len = i < 2 ? head : seg;
          const uint32_t d = tmem + 256 * (n & 1);
          if (!(ok = hold(dempty + 8 * (n & 1), (n >> 1 & 1u) ^ 1u, patient))) break;
          tc::fence_after_sync();
          uint32_t accumulate = 0;
          for (int j = min(len, left); j > 0; --j) {
            if (!there && !(ok = hold(loaded + 8 * at, parity, patient))) break;
            const uint32_t a = (ring + at * kStage) >> 4, b = a + (kABytes >> 4);
            uint64_t *const done = &sh.empty[at];
            advance<kStages>(at, parity);
            there = __all_sync(0xFFFFFFFFu, test_wait_at(loaded + 8 * at, parity)) != 0;
            tc::fence_after_sync();
            if (one) {
#pragma unroll
              for (int k = 0; k < kK / 16; ++k)
                mma_pair_ss(d, (a + 2 * k) | 1u << 16, (b + b_step * k) | b_lead, idesc, k ? 1u : accumulate);
              commit_pair(done);
            }
            __syncwarp();
            accumulate = 1;
          }
          if (ok && one) commit_pair(&sh.dfull[n & 1]);
          __syncwarp();
        }
      }
      if (one) commit_pair(&sh.drained);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    // ---------------- fold and epilogue: 32 rows, and a part of the columns in whole units of 64 (128 and 64 of
    // 192, half of 256 and 128, all or none of 64) ----------------
    const int e = warp - kEpiWarp, q = warp & 3, c = e >> 2;
    const int first = (P.bn + 127) / 128 * 64, own = c ? P.bn - first : first;   // columns of the two parts, of this warp
    uint8_t *const mine = sm + kStages * kStage + e * kBufs * kUnit;
    const uint32_t buf = tc::smem_u32(mine), lanes = tmem + ((uint32_t)(32 * q) << 16);
    constexpr int kCols = 128 / sizeof(E);           // columns of a unit
    constexpr int kPairs = Piece<E>::pairs;
    const bool one = elect_one();
    const Draw draw(P.drop);
    uint32_t n = 0, tile = 0, loads = 0, issued = 0;   // loads: buffers filled and read
    uint32_t next = buf;                               // forward: the buffer that is written next
    bool ok = true, bad = false;
    grid_wait();   // as the MMA warp
    for (int it = pair; it < P.items && ok; it += pairs, ++tile) {
      const Item w(P, it);
      const int row0 = w.m * kTileRows + 128 * rank + 32 * q, rows = P.T - row0;   // may be <= 0
      const int col0 = kGated ? 128 * w.n + 64 * c : w.n * P.bn + first * c;
      // the inputs of unit v into the warp's buffers, whose last contents have been stored
      auto load_inputs = [&](int v) {
        const int col = col0 + kCols * v;
        if (rows <= 0 || kCols * v >= own || col >= P.N) return;
        if (VEC && one) stores_read();
        __syncwarp();
        if constexpr (!VEC) {
          load_any<E>(buf, P.in0, P.T, P.N, row0, rows, col);
          if (OP == GATED_BACKWARD) load_any<E>(buf + kUnit, P.in1, P.T, P.N, row0, rows, col);
        } else if constexpr (OP == GATED_BACKWARD) {
          load_rows<E>(buf, P.in0, P.N, row0, rows, col, P.N - col);
          load_rows<E>(buf + kUnit, P.in1, P.N, row0, rows, col, P.N - col);
        } else if (one) {
          ++issued;
          load_unit(buf, &io.m[0], col, row0, tc::smem_u32(&sh.in[e]));
        }
      };
      const bool inputs = OP == GATED_BACKWARD || (OP == LINEAR && P.in0 && w.slice < 0);
      if (inputs) load_inputs(0);
      Bias<4> bias;   // forward: the gate's two and the other projection's two
      if (OP == LINEAR) {
        bias.load(P.bias0 ? P.bias0 + col0 : nullptr, min(own, P.N - col0));
      } else if (OP == GATED_FORWARD) {
        Bias<2> b0, b1;
        b0.load(P.bias0 ? P.bias0 + col0 : nullptr, P.N - col0);
        b1.load(P.bias1 ? P.bias1 + col0 : nullptr, P.N - col0);
        bias.v[0] = b0.v[0];
        bias.v[1] = b0.v[1];
        bias.v[2] = b1.v[0];
        bias.v[3] = b1.v[1];
      }
      // dropout's bits are drawn while the tile is multiplied: 16 columns each
      uint32_t keep[8];
      if (OP == LINEAR && draw.below && w.slice < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (16 * i < own) keep[i] = draw.keep16(row0 + lane, (col0 + 16 * i) / 8);
      }
      float2 acc[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] = both(0.0f);
#pragma unroll 1
      for (int left = (w.k1 - w.k0) * kTerms, i = 0; left > 0; left -= i < 2 ? P.head : P.seg, ++i, ++n) {
        if (!(ok = wait(&sh.dfull[n & 1], n >> 1 & 1u))) break;
        __syncwarp();
        tc::fence_after_sync();
        const uint32_t from = lanes + 256 * (n & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (32 * j >= own) break;
          uint32_t raw[32];
          tc::tmem_ld32_nowait(from + (kGated ? (j < 2 ? 64 * c + 32 * j : 64 + 64 * c + 32 * j) : first * c + 32 * j), raw);
          tc::tmem_wait_ld(raw);
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float2 &s = acc[2 * j + x / 16][x % 16 / 2];
            s = add2(s, make_float2(__uint_as_float(raw[x]), __uint_as_float(raw[x + 1])));
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_first(&sh.dempty[n & 1]);
      }
      if (!ok) break;

      // a buffer to its place in a tensor
      auto store = [&](uint32_t from, const CUtensorMap *map, void *to, int col) {
        if constexpr (VEC) {
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (one) store_unit(from, map, col, row0);
        } else {
          __syncwarp();
          store_any<E, kCols>(from, to, P.N, row0, rows, col, P.N - col);
          __syncwarp();
        }
      };
      // A buffer to write, whose last contents have been stored.
      auto buffer = [&]() {
        if (VEC && one) stores_read<kGated ? 1 : 0>();
        __syncwarp();
        const uint32_t b = next;
        if (kGated) next = 2 * buf + kUnit - next;
        return b;
      };
      // Unit v of 16-column groups `from` to a tensor.
      auto put = [&](const float2 (*from)[8], const CUtensorMap *map, void *to, int v) {
        const int col = col0 + kCols * v;
        if (rows <= 0 || col >= P.N) return;
        const uint32_t b = buffer();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          write_piece(piece_at(b, lane, j), pack_piece<E>(&from[kCols * v / 16 + j * kPairs / 8][j * kPairs % 8]));
        store(b, map, to, col);
      };

      if constexpr (OP == GATED_FORWARD) {
        if (P.bias0 || P.bias1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) bias.add(acc[i], i);
        }
        // g, a(g) u in g's place, u: arithmetic between the stores
        if (P.out1) {
#pragma unroll
          for (int v = 0; v < 64 / kCols; ++v) put(acc, &io.m[1], P.out1, v);
        }
        if (P.fn == GATE_SILU) gate_forward<GATE_SILU, kAccurate>(acc);
        else if (P.fn == GATE_GELU) gate_forward<GATE_GELU, kAccurate>(acc);
        else gate_forward<GATE_GELU_TANH, kAccurate>(acc);
        if (P.out1) {
#pragma unroll
          for (int v = 0; v < 64 / kCols; ++v) put(acc + 4, &io.m[2], P.out2, v);
        }
        uint8_t(&scale)[2][128] = sh.scale[tile & 1];
        uint32_t sb = 0;
        if (P.codes) {
          // A scale group is the tile's 128 columns: this warp's 64 and the other warp's; the byte grows with the amax.
          // Columns past the matrix are zeros here.
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) m = max(m, max(abs_bits(acc[i][k].x), abs_bits(acc[i][k].y)));
          sb = P.fmt == FMT_E4M3 ? act_scale_byte<FMT_E4M3>(m) : act_scale_byte<FMT_E5M2>(m);
          scale[c][32 * q + lane] = (uint8_t)sb;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.met[q]);
        }
#pragma unroll
        for (int v = 0; v < 64 / kCols; ++v) put(acc, &io.m[0], P.out0, v);
        if (P.codes) {
          if (!(ok = wait(&sh.met[q], tile & 1u))) break;
          sb = max(sb, (uint32_t)scale[c ^ 1][32 * q + lane]);
          const float inv = act_inv_scale(sb);
          if (lane < rows) {
            bad |= sb == kActBad;
            if (c == 0) P.scales[(size_t)(row0 + lane) * P.groups + w.n] = (uint8_t)sb;
          }
          if (rows <= 0 || col0 >= P.N) continue;
          const uint32_t b = buffer();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w4 = P.fmt == FMT_E4M3 ? pack_codes<FMT_E4M3>(acc[i], inv) : pack_codes<FMT_E5M2>(acc[i], inv);
            // by TMA: rows of 64 bytes in the 64-byte swizzle
            write_piece(VEC ? b + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4) : piece_at(b, lane, i), w4);
          }
          if constexpr (VEC) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (one) store_unit(b, &io.m[3], col0, row0);
          } else {
            __syncwarp();
            store_any<uint8_t, 64>(b, P.codes, P.N, row0, rows, col0, P.N - col0);
            __syncwarp();
          }
        }
      } else if constexpr (OP == GATED_BACKWARD) {
        auto walk = [&](auto fn_c) {
          constexpr int FN = decltype(fn_c)::value;
#pragma unroll
          for (int v = 0; v < 128 / kCols; ++v) {
            const int col = col0 + kCols * v;
            if (kCols * v >= own || rows <= 0 || col >= P.N) break;
            if (VEC) loads_done();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t at = piece_at(buf, lane, j);
              const Piece<E> g(read_piece(at)), u(read_piece(at + kUnit));
              float2 *d = &acc[kCols * v / 16 + j * kPairs / 8][j * kPairs % 8], du[kPairs];
              gate_backward<FN, kAccurate, kPairs>(d, du, g.v, u.v);
              write_piece(at, pack_piece<E>(d));
              write_piece(at + kUnit, pack_piece<E>(du));
            }
            store(buf, &io.m[2], P.out0, col);
            store(buf + kUnit, &io.m[3], P.out1, col);
            load_inputs(v + 1);
          }
        };
        if (P.fn == GATE_SILU) walk(std::integral_constant<int, GATE_SILU>());
        else if (P.fn == GATE_GELU) walk(std::integral_constant<int, GATE_GELU>());
        else walk(std::integral_constant<int, GATE_GELU_TANH>());
      } else if (w.slice >= 0) {
        const int at = 128 * rank + 32 * q + lane;   // row of the tile
        float *p = P.part + (((size_t)w.at * P.slices + w.slice) * kTileRows + at) * P.bn + col0 - w.n * P.bn;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (16 * i < own && lane < rows) store_own(p + 16 * i, acc[i]);
      } else {
        if (P.bias0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (16 * i < own) bias.add(acc[i], i);
        }
        if (draw.below) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (16 * i < own) drop16(draw, acc[i], keep[i]);
        }
#pragma unroll
        for (int v = 0; v < 128 / kCols; ++v) {
          const int col = col0 + kCols * v;
          if (kCols * v >= own || rows <= 0 || col >= P.N) break;
          if (inputs) {
            if (VEC) {
              if (!(ok = wait(&sh.in[e], loads & 1u))) break;
              ++loads;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const Piece<E> r(read_piece(piece_at(buf, lane, j)));
              float2 *x = &acc[kCols * v / 16 + j * kPairs / 8][j * kPairs % 8];
#pragma unroll
              for (int k = 0; k < kPairs; ++k) x[k] = add2(x[k], r.v[k]);
            }
          }
          put(acc, &io.m[2], P.out0, v);
          if (inputs) load_inputs(v + 1);
        }
      }
    }
    // nothing of this warp's is in flight when the CTA leaves: its stores, and loads whose wait did not end
    if (one) {
      stores_done();
      if (issued != loads) tc::mbar_wait_bounded(&sh.in[e], loads & 1u, kDrain);
    }
    if (OP == GATED_BACKWARD) loads_done();
    if (bad) set_status(status, GIFT_ERR_NONFINITE);
  }

  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();   // the peer no longer arrives on this CTA's barriers, and its MMAs are done
  const uint32_t most = max(max(sh.issued[0], sh.issued[1]), max(sh.issued[2], sh.issued[3]));
  if (most & kGaveUp) {   // the same in both CTAs
    // The copies that were made land on the first CTA's barriers: it arrives for those that were not, and waits.
    if (rank == 0 && tid == 0) {
      uint32_t g = 0;
      for (int i = 0; i < 4; ++i) g = max(g, sh.issued[i] & ~kGaveUp);
      for (int i = 0; i < 4; ++i)
        for (uint32_t u = sh.issued[i] & ~kGaveUp; u < g; ++u) tc::mbar_arrive(&sh.full[u % kStages]);
      landed<kStages>(sh.full, g);
    }
    __syncwarp();   // the cluster barrier and the dealloc below are for converged warps
    cluster_sync();
  }
  if (warp == 0) {
    tc::fence_after_sync();
    dealloc_pair(tmem);
  }
}

template <int OP, typename E, bool VEC, bool MN>
cudaError_t launch(const Launch &L, const Params &P, const CUtensorMap *maps, const IoMaps &io, int pairs, bool after) {
  const cudaError_t e = ensure_dynamic_smem<k_product<OP, E, VEC, MN>>(Cfg<OP>::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (P.items < pairs ? P.items : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<OP>::smem;
  cfg.stream = L.stream;
  // `after` the launch that makes the operands, itself ordered behind everything before it: this one may
  // start beside it (grid_wait).  Without that launch the kernel waits for its predecessors as usual.
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_product<OP, E, VEC, MN>, P, maps[0], maps[1], maps[2], maps[3], io,
                            L.status);
}

template <int OP, bool MN>
cudaError_t launch_typed(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                         const IoMaps &io, int pairs, bool after) {
  if (bf16)
    return vec ? launch<OP, __nv_bfloat16, true, MN>(L, P, maps, io, pairs, after)
               : launch<OP, __nv_bfloat16, false, MN>(L, P, maps, io, pairs, after);
  return vec ? launch<OP, float, true, MN>(L, P, maps, io, pairs, after)
             : launch<OP, float, false, MN>(L, P, maps, io, pairs, after);
}

// One launch per file, so that they compile side by side.
cudaError_t launch_gated_forward(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                                 const IoMaps &io, int pairs, bool after);
cudaError_t launch_gated_backward(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                                  const IoMaps &io, int pairs, bool after);
cudaError_t launch_linear(const Launch &L, bool bf16, bool vec, bool mn, const Params &P, const CUtensorMap *maps,
                          const IoMaps &io, int pairs, bool after);
cudaError_t launch_linear_mn(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                             const IoMaps &io, int pairs, bool after);

}  // namespace product

}  // namespace gift
