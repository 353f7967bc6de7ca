// The feed-forward block's products on the 5th-generation tensor cores: one persistent kernel, its epilogue by
// operator.  out[t][n] = sum_k A[t][k] B[k][n], A the T tokens' rows (K contiguous), B a weight matrix read as it
// lies in memory, K-major (n x k: a forward product) or MN-major (k x n: a product with its transpose).
//
// A pair of CTAs (a cluster of two SMs, cta_group::2) owns 256 tokens x up to 256 columns: each CTA holds 128 of
// the tokens and half of B's columns.  Per CTA:
//   warp 0       TMA: stages of 64 k, A's 128 x 64 and B's up to 128 x 64 elements;
//   warp 1       the pair's first CTA issues 256 x N x 16 MMAs; the second one's reports its stages to the first;
//   warps 4-11   fold and epilogue: a thread has one token and half of the tile's columns.
// The tensor core truncates its sums, so a segment of at most 512 k goes into one of two accumulators in tensor
// memory and is added to FP32 registers to nearest while the other is filled.  The epilogue runs from those
// registers while the next tile's first two segments are multiplied.
// The gated forward product takes its two projections as one product of 128 + 128 columns: the first CTA loads
// the gate's rows, the second the other projection's, and both halves of a row meet in one thread.
// FP32 operands are three BF16 terms each (operand.cuh); a block of 64 k then takes six stages, the products i + j <= 2
// of terms i and j; what is dropped is below 2^-23 of |A_k B_k|.  A block is a segment and the small products come
// first, so that only the last stage's four steps truncate at the sum's size (segments of two blocks: outputs 6e-7
// off instead of 2e-7 at 256 k).
// Every mbarrier wait is bounded by the context's GIFT_OPT_BARRIER_WAIT and reports GIFT_ERR_TIMEOUT; a warp
// leaves as one, and the copies and MMAs in flight are waited for before the CTA leaves.
#pragma once

#include <type_traits>

#include "act.cuh"
#include "dropout.cuh"
#include "gate.cuh"
#include "kernels.cuh"
#include "pair.cuh"

namespace gift {

namespace product {

constexpr int kK = 64;                      // k of a stage
constexpr int kABytes = 128 * kK * 2;       // a CTA's rows of A in a stage, and its most columns of B
constexpr int kStage = 2 * kABytes;
constexpr int kStages = 6;
constexpr int kBox = kK * 128;              // bytes of an MN-major box: 64 columns
constexpr int kThreads = 384;
constexpr int kEpiWarp = 4, kEpiWarps = 8;
constexpr int kTileRows = 256;
constexpr int kPitch = 17;                  // floats of a row of the epilogue's 32 x 16 staging tiles
constexpr int kSmem = kStages * kStage + kEpiWarps * 32 * kPitch * 4 + 1024;

enum Op { GATED_FORWARD, GATED_BACKWARD, LINEAR, SLICE };

struct Params {
  int T, N;               // rows and columns of the output
  int mt, nt, slices, items;
  int kb, kb1;            // blocks of 64 k, and those of the first pair of operands
  int terms;              // products per block: 1, or 6 of FP32's terms
  int seg;                // stages of a segment
  int bn;                 // columns of a tile, a multiple of 64
  int b_mn;               // B is MN-major
  uint32_t idesc;
  long long budget;       // clocks of a wait
  // epilogue
  int fn, fmt, groups;
  const float *bias0, *bias1;   // nullable
  const void *in0, *in1;        // gated backward: gate, up; linear: in0 the residual (nullable)
  void *out0, *out1, *out2;     // forward: h, gate, up (nullable both); backward: dgate, dup; linear: y
  uint8_t *codes, *scales;      // nullable: h's 8-bit checkpoint
  Dropout drop;
  float *part;                  // slices: [slices][T][part_ld]
  int part_ld;
};

struct Item {
  int m, n, slice, k0, k1;   // tile, blocks of 64 k
  // Tiles in groups of eight rows of tiles, column by column within a group: the pairs that run at the same time
  // share both operands in L2.
  __device__ __forceinline__ Item(const Params &P, int item) {
    const int tiles = P.mt * P.nt, tile = item % tiles;
    slice = item / tiles;
    const int per = 8 * P.nt, g = tile / per, rem = tile - g * per, rows = min(8, P.mt - 8 * g);
    n = rem / rows;
    m = 8 * g + rem - n * rows;
    k0 = (int)((long long)P.kb * slice / P.slices);
    k1 = (int)((long long)P.kb * (slice + 1) / P.slices);
  }
};

struct __align__(16) Shared {
  uint64_t full[kStages], empty[kStages];   // loaded; multiplied (in both CTAs)
  uint64_t other[kStages];                  // first CTA: the second one's stage is loaded
  uint64_t dfull[2], dempty[2];             // accumulators: summed; folded by both CTAs
  uint64_t met[4];                          // a row's two column halves have left their amax
  uint64_t drained;
  uint32_t amax[2][2][128];                 // [tile parity][half][row]
  uint32_t tmem;
  volatile int failed;
};

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

// ---- a thread's 16 columns of one row, of 32 consecutive rows per warp ---------------------------------
// VEC: rows of a multiple of 16 elements in 32-byte aligned buffers; a lane moves its own row's columns.  Otherwise
// through the warp's staging tile, so that 16 lanes move 16 consecutive columns.
template <typename E, bool VEC>
struct Cols;
template <>
struct Cols<__nv_bfloat16, true> {
  uint32_t r[8];
  __device__ __forceinline__ void load(const void *base, size_t ld, int row0, int rows, int col, int n, float *) {
    const int lane = threadIdx.x & 31;
    if (lane < rows && n > 0) ld256(static_cast<const __nv_bfloat16 *>(base) + (size_t)(row0 + lane) * ld + col, r);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = 0u;
  }
  __device__ __forceinline__ float2 pair(int k) const {
    return make_float2(__uint_as_float(r[k] << 16), __uint_as_float(r[k] & 0xFFFF0000u));
  }
};
template <>
struct Cols<float, true> {
  uint32_t r[16];
  __device__ __forceinline__ void load(const void *base, size_t ld, int row0, int rows, int col, int n, float *) {
    const int lane = threadIdx.x & 31;
    if (lane < rows && n > 0) {
      const float *p = static_cast<const float *>(base) + (size_t)(row0 + lane) * ld + col;
      ld256(p, r);
      ld256(p + 8, r + 8);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) r[e] = 0u;
    }
  }
  __device__ __forceinline__ float2 pair(int k) const {
    return make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
  }
};
template <typename E>
struct Cols<E, false> {
  float2 v[8];
  __device__ __forceinline__ void load(const void *base, size_t ld, int row0, int rows, int col, int n, float *stage) {
    const int lane = threadIdx.x & 31, c = lane & 15;
    const E *p = static_cast<const E *>(base) + (size_t)row0 * ld + col + c;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = 2 * k + (lane >> 4);
      stage[r * kPitch + c] = r < rows && c < n ? ld1(p + (size_t)r * ld) : 0.0f;
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = make_float2(stage[lane * kPitch + 2 * k], stage[lane * kPitch + 2 * k + 1]);
    __syncwarp();
  }
  __device__ __forceinline__ float2 pair(int k) const { return v[k]; }
};

template <typename E, bool VEC>
__device__ __forceinline__ void store16(void *base, size_t ld, int row0, int rows, int col, int n, const float2 *v,
                                        float *stage) {
  const int lane = threadIdx.x & 31;
  E *p = static_cast<E *>(base) + (size_t)row0 * ld + col;
  if (VEC) {
    if (lane < rows && n > 0) {
      p += (size_t)lane * ld;
      if constexpr (sizeof(E) == 2) {
        uint32_t r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = pack_bf16(v[k].x, v[k].y);
        st256(p, r);
      } else {
        uint32_t r[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          r[2 * k] = __float_as_uint(v[k].x);
          r[2 * k + 1] = __float_as_uint(v[k].y);
        }
        st256(p, r);
        st256(p + 8, r + 8);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      stage[lane * kPitch + 2 * k] = v[k].x;
      stage[lane * kPitch + 2 * k + 1] = v[k].y;
    }
    __syncwarp();
    const int c = lane & 15;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = 2 * k + (lane >> 4);
      if (r < rows && c < n) st1(p + (size_t)r * ld + c, stage[r * kPitch + c]);
    }
    __syncwarp();
  }
}

// 16 codes of a row: VEC as above (and 16-byte aligned codes)
template <int F, bool VEC>
__device__ __forceinline__ void store_codes(uint8_t *base, size_t ld, int row0, int rows, int col, int n,
                                            const float2 *v, float inv, float *stage) {
  const int lane = threadIdx.x & 31;
  const float2 s = both(inv);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = mul2(v[2 * k], s), b = mul2(v[2 * k + 1], s);
    w[k] = pack4_fp8<F>(a.x, a.y, b.x, b.y);
  }
  uint8_t *p = base + (size_t)row0 * ld + col;
  if (VEC) {
    if (lane < rows && n > 0) *reinterpret_cast<uint4 *>(p + (size_t)lane * ld) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t *t = reinterpret_cast<uint32_t *>(stage);   // rows of 5 words: 20 bytes
#pragma unroll
    for (int k = 0; k < 4; ++k) t[lane * 5 + k] = w[k];
    __syncwarp();
    const uint8_t *b = reinterpret_cast<const uint8_t *>(stage);
    const int c = lane & 15;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = 2 * k + (lane >> 4);
      if (r < rows && c < n) p[(size_t)r * ld + c] = b[r * 20 + c];
    }
    __syncwarp();
  }
}

// bias of 16 columns (the same for every lane), n of them in the matrix; nullable
__device__ __forceinline__ void add_bias(float2 *v, const float *bias, int n) {
  if (!bias) return;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    v[k] = add2(v[k], make_float2(2 * k < n ? bias[2 * k] : 0.0f, 2 * k + 1 < n ? bias[2 * k + 1] : 0.0f));
}

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
// dh in `d`: the gate's gradient in its place, the other projection's in `du`
template <int FN, bool ACCURATE, typename C>
__device__ __forceinline__ void gate_backward(float2 *d, float2 *du, const C &g, const C &u) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 gv = g.pair(k);
    float2 slope, a;
    a.x = gate_slope<FN, ACCURATE>(gv.x, slope.x);
    a.y = gate_slope<FN, ACCURATE>(gv.y, slope.y);
    du[k] = mul2(d[k], a);
    d[k] = mul2(mul2(d[k], u.pair(k)), slope);
  }
}

template <int OP, typename E, bool VEC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_product(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap tm_a0,
              const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b0,
              const __grid_constant__ CUtensorMap tm_b1, int *status) {
  constexpr bool kGated = OP == GATED_FORWARD;
  constexpr bool kAccurate = sizeof(E) == 4;
  extern __shared__ uint8_t dsm[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(((uintptr_t)dsm + 1023) & ~(uintptr_t)1023);
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (OP == SLICE) grid_release();   // the kernel that joins the slices

  if (warp == 0) alloc_pair(&sh.tmem);
  if (tid == 32) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&sh.full[s], 1);
      tc::mbar_init(&sh.empty[s], 1);
      tc::mbar_init(&sh.other[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&sh.dfull[b], 1);
      tc::mbar_init(&sh.dempty[b], 2 * kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) tc::mbar_init(&sh.met[q], 2);
    tc::mbar_init(&sh.drained, 1);
    tc::fence_mbar_init();
    sh.failed = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  // Called by whole warps: the lanes go on together, or none does.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    bool done = tc::mbar_try_wait(bar, parity);
    if (!done) {
      const long long t0 = clock64();
      do {
        if (sh.failed || clock64() - t0 > P.budget) {
          sh.failed = 1;
          set_status(status, GIFT_ERR_TIMEOUT);
          break;
        }
        done = tc::mbar_try_wait(bar, parity);
      } while (!done);
    }
    return __all_sync(0xFFFFFFFFu, done) != 0;
  };

  // registers: 168 per thread at launch (504 over the three groups of four warps), redistributed as 2 x 208 + 88
  if (warp < kEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    const bool one = elect_one();
    if (warp == 0) {
      // ---------------- TMA ----------------
      const int half = P.bn / 2, boxes = (half + 63) / 64;
      const uint32_t bytes = kABytes + (P.b_mn ? boxes * kBox : half * 128);
      uint32_t g = 0;
      bool ok = true;
      grid_wait();   // the operands that the launch before this one made
      for (int it = pair; it < P.items && ok; it += pairs) {
        const Item w(P, it);
        const int row = w.m * kTileRows + 128 * rank;
        const int col = kGated ? 128 * w.n : w.n * P.bn + half * rank;
        const CUtensorMap *gate = rank ? &tm_b1 : &tm_b0;
        for (int kb = w.k0; kb < w.k1 && ok; ++kb) {
          const bool second = !kGated && kb >= P.kb1;
          const int k = (second ? kb - P.kb1 : kb) * kK;
          const CUtensorMap *a = second ? &tm_a1 : &tm_a0, *b = kGated ? gate : second ? &tm_b1 : &tm_b0;
          for (int p = 6 - P.terms; p < 6; ++p, ++g) {   // terms (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
            const int ta = (0x001012 >> (4 * p)) & 3, tb = (0x010210 >> (4 * p)) & 3;
            const Slot<kStages> s(g);
            if (!(ok = wait(&sh.empty[s.at], s.parity ^ 1u))) break;
            if (one) {
              uint8_t *st = sm + s.at * kStage;
              tc::mbar_arrive_expect_tx(&sh.full[s.at], bytes);
              tma_load_3d(st, a, k, row, ta, &sh.full[s.at]);
              if (P.b_mn) {
                for (int x = 0; x < boxes; ++x)
                  tma_load_3d(st + kABytes + x * kBox, b, col + 64 * x, k, tb, &sh.full[s.at]);
              } else {
                tma_load_3d(st + kABytes, b, k, col, tb, &sh.full[s.at]);
              }
            }
          }
        }
      }
      // leave no arrival of the MMAs' commits behind: the last stages'
      for (uint32_t r = 1; ok && r <= kStages && r <= g; ++r) {
        const Slot<kStages> s(g - r);
        ok = wait(&sh.empty[s.at], s.parity);
      }
      landed<kStages>(sh.full, g);
      // the pair's first CTA may have a wait of its own to end before its last commit
      tc::mbar_wait_bounded(&sh.drained, 0, P.budget + kDrain);
    } else if (warp == 1 && rank == 0) {
      // ---------------- MMA ----------------
      const uint32_t first = tc::smem_u32(sm) >> 4;
      const uint32_t b_lead = P.b_mn ? (uint32_t)(kBox >> 4) << 16 : 1u << 16, b_step = P.b_mn ? 128u : 2u;
      uint32_t g = 0, n = 0;   // stages, segments
      bool ok = true;
      for (int it = pair; it < P.items && ok; it += pairs) {
        const Item w(P, it);
        for (int left = (w.k1 - w.k0) * P.terms; left > 0 && ok; left -= P.seg, ++n) {
          const uint32_t d = tmem + 256 * (n & 1);
          if (!(ok = wait(&sh.dempty[n & 1], (n >> 1 & 1u) ^ 1u))) break;
          tc::fence_after_sync();
          for (int j = 0; j < P.seg && j < left; ++j, ++g) {
            const Slot<kStages> s(g);
            if (!(ok = wait(&sh.full[s.at], s.parity) && wait(&sh.other[s.at], s.parity))) break;
            tc::fence_after_sync();
            if (one) {
              const uint32_t a = first + s.at * (kStage >> 4), b = a + (kABytes >> 4);
#pragma unroll
              for (int k = 0; k < kK / 16; ++k)
                mma_pair_ss(d, (a + 2 * k) | 1u << 16, (b + b_step * k) | b_lead, P.idesc, j || k ? 1u : 0u);
              commit_pair(&sh.empty[s.at]);
            }
          }
          if (ok && one) commit_pair(&sh.dfull[n & 1]);
        }
      }
      if (one) commit_pair(&sh.drained);
    } else if (warp == 1) {
      // ---------------- the second CTA's stages ----------------
      uint32_t total = 0;
      for (int it = pair; it < P.items; it += pairs) {
        const Item w(P, it);
        total += (uint32_t)(w.k1 - w.k0) * P.terms;
      }
      for (uint32_t g = 0; g < total; ++g) {
        const Slot<kStages> s(g);
        if (!wait(&sh.full[s.at], s.parity)) break;
        if (one) arrive_first(&sh.other[s.at]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    // ---------------- fold and epilogue: 32 rows, half of the columns ----------------
    const int q = warp & 3, c = (warp - kEpiWarp) >> 2;
    const int half = P.bn / 2;
    float *stage = reinterpret_cast<float *>(sm + kStages * kStage) + (warp - kEpiWarp) * 32 * kPitch;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    const Draw draw(P.drop);
    uint32_t n = 0, tile = 0;
    bool ok = true, bad = false;
    for (int it = pair; it < P.items && ok; it += pairs, ++tile) {
      const Item w(P, it);
      const int row0 = w.m * kTileRows + 128 * rank + 32 * q, rows = P.T - row0;   // may be <= 0
      float2 acc[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] = both(0.0f);
#pragma unroll 1
      for (int left = (w.k1 - w.k0) * P.terms; left > 0; left -= P.seg, ++n) {
        if (!(ok = wait(&sh.dfull[n & 1], n >> 1 & 1u))) break;
        tc::fence_after_sync();
        const uint32_t from = lanes + 256 * (n & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (32 * j >= half) break;
          uint32_t raw[32];
          tc::tmem_ld32_nowait(from + (kGated ? (j < 2 ? 64 * c + 32 * j : 64 + 64 * c + 32 * j) : half * c + 32 * j), raw);
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

      if constexpr (OP == GATED_FORWARD) {
        const int f0 = 128 * w.n + 64 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = f0 + 16 * i, left = P.N - col;
          add_bias(acc[i], P.bias0 ? P.bias0 + col : nullptr, left);
          add_bias(acc[4 + i], P.bias1 ? P.bias1 + col : nullptr, left);
          if (P.out1) {
            store16<E, VEC>(P.out1, P.N, row0, rows, col, left, acc[i], stage);
            store16<E, VEC>(P.out2, P.N, row0, rows, col, left, acc[4 + i], stage);
          }
        }
        if (P.fn == GATE_SILU) gate_forward<GATE_SILU, kAccurate>(acc);
        else if (P.fn == GATE_GELU) gate_forward<GATE_GELU, kAccurate>(acc);
        else gate_forward<GATE_GELU_TANH, kAccurate>(acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store16<E, VEC>(P.out0, P.N, row0, rows, f0 + 16 * i, P.N - f0 - 16 * i, acc[i], stage);
        if (P.codes) {
          // a scale group is the tile's 128 columns: this warp's 64 and the other half's
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (f0 + 16 * i + 2 * k < P.N) {   // columns past the matrix are not its last group's
                m = max(m, abs_bits(acc[i][k].x));
                if (f0 + 16 * i + 2 * k + 1 < P.N) m = max(m, abs_bits(acc[i][k].y));
              }
          uint32_t(&amax)[2][128] = sh.amax[tile & 1];
          amax[c][32 * q + lane] = m;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.met[q]);
          if (!(ok = wait(&sh.met[q], tile & 1u))) break;
          m = max(m, amax[c ^ 1][32 * q + lane]);
          const uint32_t sb = P.fmt == FMT_E4M3 ? act_scale_byte<FMT_E4M3>(m) : act_scale_byte<FMT_E5M2>(m);
          const float inv = act_inv_scale(sb);
          if (lane < rows) {
            bad |= sb == kActBad;
            if (c == 0) P.scales[(size_t)(row0 + lane) * P.groups + w.n] = (uint8_t)sb;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int col = f0 + 16 * i, left = P.N - col;
            if (P.fmt == FMT_E4M3)
              store_codes<FMT_E4M3, VEC>(P.codes, P.N, row0, rows, col, left, acc[i], inv, stage);
            else
              store_codes<FMT_E5M2, VEC>(P.codes, P.N, row0, rows, col, left, acc[i], inv, stage);
          }
        }
      } else if constexpr (OP == GATED_BACKWARD) {
        auto walk = [&](auto fn_c) {
          constexpr int FN = decltype(fn_c)::value;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (16 * i >= half) break;
            const int col = w.n * P.bn + half * c + 16 * i, left = P.N - col;
            Cols<E, VEC> g, u;
            g.load(P.in0, P.N, row0, rows, col, left, stage);
            u.load(P.in1, P.N, row0, rows, col, left, stage);
            float2 du[8];
            gate_backward<FN, kAccurate>(acc[i], du, g, u);
            store16<E, VEC>(P.out0, P.N, row0, rows, col, left, acc[i], stage);
            store16<E, VEC>(P.out1, P.N, row0, rows, col, left, du, stage);
          }
        };
        if (P.fn == GATE_SILU) walk(std::integral_constant<int, GATE_SILU>());
        else if (P.fn == GATE_GELU) walk(std::integral_constant<int, GATE_GELU>());
        else walk(std::integral_constant<int, GATE_GELU_TANH>());
      } else if constexpr (OP == LINEAR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (16 * i >= half) break;
          const int col = w.n * P.bn + half * c + 16 * i, left = P.N - col;
          add_bias(acc[i], P.bias0 ? P.bias0 + col : nullptr, left);
          if (draw.below) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t keep = draw.keep8(row0 + lane, col / 8 + h);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float2 &v = acc[i][4 * h + k];
                v.x = keep >> (2 * k) & 1u ? v.x * draw.scale : 0.0f;
                v.y = keep >> (2 * k + 1) & 1u ? v.y * draw.scale : 0.0f;
              }
            }
          }
          if (P.in0) {
            Cols<E, VEC> r;
            r.load(P.in0, P.N, row0, rows, col, left, stage);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[i][k] = add2(acc[i][k], r.pair(k));
          }
          store16<E, VEC>(P.out0, P.N, row0, rows, col, left, acc[i], stage);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (16 * i >= half) break;
          const int col = w.n * P.bn + half * c + 16 * i;
          store16<float, true>(P.part + (size_t)w.slice * P.T * P.part_ld, P.part_ld, row0, rows, col,
                               P.part_ld - col, acc[i], stage);
        }
      }
    }
    if (bad) set_status(status, GIFT_ERR_NONFINITE);
  }

  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();   // the peer no longer arrives on this CTA's barriers, and its MMAs are done
  if (warp == 0) {
    tc::fence_after_sync();
    dealloc_pair(tmem);
  }
}

template <int OP, typename E, bool VEC>
cudaError_t launch(const Launch &L, const Params &P, const CUtensorMap *maps, int pairs, bool after) {
  const cudaError_t e = ensure_dynamic_smem<k_product<OP, E, VEC>>(kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (P.items < pairs ? P.items : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = L.stream;
  // `after` the launch that makes the operands, itself ordered behind everything before it: this one may
  // start beside it (grid_wait).  Without that launch the kernel waits for its predecessors as usual.
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_product<OP, E, VEC>, P, maps[0], maps[1], maps[2], maps[3], L.status);
}

template <int OP>
cudaError_t launch_typed(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps, int pairs,
                         bool after) {
  if (bf16)
    return vec ? launch<OP, __nv_bfloat16, true>(L, P, maps, pairs, after)
               : launch<OP, __nv_bfloat16, false>(L, P, maps, pairs, after);
  return vec ? launch<OP, float, true>(L, P, maps, pairs, after) : launch<OP, float, false>(L, P, maps, pairs, after);
}

// One launch per file, so that they compile side by side.
cudaError_t launch_gated_forward(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                                 int pairs, bool after);
cudaError_t launch_gated_backward(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps,
                                  int pairs, bool after);
cudaError_t launch_linear(const Launch &L, bool bf16, bool vec, const Params &P, const CUtensorMap *maps, int pairs,
                          bool after);
cudaError_t launch_slices(const Launch &L, const Params &P, const CUtensorMap *maps, int pairs, bool after);

}  // namespace product

}  // namespace gift
