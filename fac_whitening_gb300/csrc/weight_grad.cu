// Weight gradient from an 8-bit checkpoint, dW = delta^T v, on the 5th-generation tensor cores.
//
// dW[o][i] = sum_t delta[t][o] v[t][i] contracts over tokens, the slow axis of both operands.  The
// kernel forms D[i][o] with the checkpoint as the A operand in tensor memory (M = i) and delta as
// the B operand in shared memory (N = o, read MN-major as TMA wrote it: no transposed copy of
// either).  A value code * 2^k is exact in BF16, so the products are exact and the only roundings
// are the sums'.
//
// A pair of CTAs (a cluster of two SMs, cta_group::2) owns a 256 (i) x 128 NH (o) tile and walks
// its tokens 64 at a time; each CTA holds 128 of the i and half of the o columns:
//   warps 0, 2   TMA: a stage's 64 x 128 code tile and its tokens' scales (one group of 128 columns:
//                the CTA's; transposed and made BF16 by k_prepare); its 64 x 64 delta boxes;
//   warps 4-19   codes -> BF16: ldmatrix transposes 16 x 16 bytes so that a register holds four
//                tokens of one column, which is tcgen05.st's 16x256b layout; the code's bits placed
//                in the BF16 fields times 2^(120 + k) (2^(112 + k) for E5M2), exact;
//   warps 1, 3   the pair's first CTA issues 256 x 128 x 16 MMAs, a warp for each half of the tile;
//   warps 20-27  fold: the tensor core truncates its sums, so a segment of at most 256 tokens goes
//                into one of three 128-column accumulators and is added to FP32 registers to
//                nearest; the two halves of a tile change accumulators half a segment apart, so
//                that one is always being drained while two are being filled.
// Few tiles: the tokens are cut into slices whose sums a second kernel adds in order.  db is the row
// that a value of 1 for every token gives: a group of ones after the last columns (plan_for).
//
// What bounds it.  The MMAs take 512 clocks a stage (measured back to back, N = 128 halves as well as
// N = 256).  One CTA alone would need 80 bytes of operands per clock from L2, a pair needs 48 per SM.
// The conversion costs the SM's integer pipes about 250 clocks a stage, and every warp's waits and
// issues around it are latency: the numbers of warps, the two rings and the two MMA warps come from
// there.  16384 x 1536 x 6144 (tokens x d_out x d_in): 185 us for this kernel with cold caches, 1.67
// PFLOP/s (a call 193 us alone, 212 to 219 in passes one after the other); 65536 tokens 712 to 724 us a
// call, 1.72 PFLOP/s; 32768 x 4096 x 16384 run over and over (power cap) 3.0 to 3.1 ms, 1.42 to 1.46
// PFLOP/s; FP32 delta 16384 x 1536 x 6144 with db 522 us a call, 0.94 of its threefold products at the
// measured rate.  Converting in a pass of its own would move 300 MB more for the first of these, 45 us
// at the copy rate.
// The 72 registers of a launch spill 52 bytes stored and 116 loaded for BF16, 144 and 148 for FP32 delta
// (two halves).
// Every mbarrier wait is bounded by the context's GIFT_OPT_BARRIER_WAIT and reports GIFT_ERR_TIMEOUT.  A
// warp leaves as one, and however its loop ended, the copies it issued and the MMAs on the CTA's
// memory are waited for before the CTA leaves.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "act.cuh"
#include "kernels.cuh"
#include "tc.cuh"

namespace gift {

namespace {

constexpr int kK = 64;                       // tokens of a stage
constexpr int kBox = kK * 128;               // bytes of one 128-byte-wide box: codes, or 64 BF16 columns
constexpr int kGroup = 4;                    // stages of a group, and A operand slots in tensor memory
                                             // (32 columns each): stage j of a group uses slot j
constexpr int kACol = 384;                   // after three 128-column accumulators
constexpr int kFoldWarps = 8;                // warps 20-27
constexpr int kDeqWarp = 4, kDeqWarps = 16;  // warps 4-19: four per stage, by turns
constexpr int kFoldWarp = kDeqWarp + kDeqWarps;
constexpr int kCodesWarp = 0, kMmaWarp = 1, kDeltaWarp = 2;   // and the second half's MMA warp, 3
constexpr int kThreads = 896;
constexpr long long kDrain = 4000000000LL;   // clocks that a leaving warp waits for what is in flight, about 2 s

// Two rings in shared memory.  A code box is free as soon as it is converted; delta's boxes are held
// until their MMAs are done, up to four stages later.  So delta gets the deeper part of the 224 KB:
// with one ring of eight stages for both, four were left for loads in flight (65536 x 1536 x 6144: 818
// us with one ring, 790 with two and a TMA warp for each; one TMA warp for both took 1030).
template <int NH, int TERMS>
struct Cfg {
  static constexpr int delta_bytes = kBox * NH * TERMS;       // of a stage
  static constexpr int codes = TERMS == 1 ? (NH == 2 ? 8 : 12) : (NH == 2 ? 4 : 8);   // a multiple of kGroup
  static constexpr int deltas = TERMS == 1 ? (NH == 2 ? 10 : 14) : (NH == 2 ? 4 : 6);
  static constexpr int period = TERMS == 1 ? 4 : 2;           // stages of a segment: at most 256 tokens
  static constexpr int smem = codes * kBox + deltas * delta_bytes + 1024;
};

// What a stage's conversion reads: for each token t of the group, its scale 2^k times 2^120 (2^112)
// as BF16, cut off at 2^127; the exponent that was cut off (0 for activations below 448 * 2^7 or
// 57344 * 2^15), and whether any was.
struct StageScales {
  uint16_t first[kK];
  uint8_t over[kK];
  uint32_t any_over, pad[3];
};
constexpr int kScaleBytes = sizeof(StageScales);

// The kernel's static shared memory: 2048 bytes for two halves of BF16 delta, which is all that its rings leave.
template <int NH, int TERMS>
struct __align__(16) Shared {
  using C = Cfg<NH, TERMS>;
  StageScales scales[C::codes];
  uint64_t cfull[C::codes], cempty[C::codes];     // codes with their scales: loaded, converted
  uint64_t bfull[C::deltas], bempty[C::deltas];   // delta: loaded, multiplied
  uint64_t ready[kGroup];                         // A slot: converted in both CTAs
  uint64_t dfull[3], dempty[3];                   // accumulators: summed, folded
  uint64_t drained;                               // every MMA issued is done
  uint32_t tmem;
  volatile int failed;
};

struct Params {
  int T, d_out, d_in, last_group;
  int ng;                      // groups of stages (256 tokens) over all tokens; tokens past T are zeros
  int mt, nt, slices, items;
  const StageScales *scales;   // last_group + 1 rows of `stages`
  int stages;
  const float *gamma;          // nullable
  float *out;                  // dW, or the slices' sums (slice s at s d_out d_in)
  int ones;                    // the row whose values are 1 (-1: none)
  const uint8_t *one_codes;    // a box of the code of 1
  float *db;                   // where that row's sums go
  long long budget;            // clocks of a wait
};

// One work item: an output tile and a range of groups.
struct Item {
  int i0, o0, slice, t0, ng;
  __device__ __forceinline__ Item(const Params &P, int item, int on) {
    const int tiles = P.mt * P.nt, tile = item % tiles;
    slice = item / tiles;
    i0 = tile % P.mt * 256;
    o0 = tile / P.mt * on;
    const int g0 = (int)((long long)P.ng * slice / P.slices);
    t0 = g0 * (kGroup * kK);
    ng = (int)((long long)P.ng * (slice + 1) / P.slices) - g0;
  }
};

// Which of the three 128-column accumulators each half of the tile is summed in.  A half that
// starts a segment takes the one that has been free longest; the MMA warp and the fold warps each
// keep one of these and see the same sequence.
template <int NH>
struct Accumulators {
  int cur0 = NH == 2 ? 1 : 2, cur1 = 2, spare = 0;
  uint32_t phase = 0;   // bit b: uses of accumulator b so far, mod 2
  __device__ __forceinline__ void start_tile() {
    if (NH == 2) {
      const int t = spare;
      spare = cur1;
      cur1 = cur0;
      cur0 = t;
    } else {
      next(0);
    }
  }
  __device__ __forceinline__ void next(int h) {
    if (NH == 1) {
      cur0 = cur0 == 2 ? 0 : cur0 + 1;
    } else if (h == 0) {
      const int t = cur0;
      cur0 = spare;
      spare = t;
    } else {
      const int t = cur1;
      cur1 = spare;
      spare = t;
    }
  }
  __device__ __forceinline__ int cur(int h) const { return h == 0 ? cur0 : cur1; }
  // what the next change takes
  __device__ __forceinline__ int upcoming() const { return NH == 2 ? spare : cur0 == 2 ? 0 : cur0 + 1; }
  // the parity of accumulator b's current use, counted
  __device__ __forceinline__ uint32_t use(int b) {
    const uint32_t par = (phase >> b) & 1u;
    phase ^= 1u << b;
    return par;
  }
};

// The slot of a ring of N that its g-th use takes, and the parity of that use.
template <int N>
struct Slot {
  uint32_t at, parity;
  __device__ __forceinline__ explicit Slot(uint32_t g) : at(g % N), parity(g / N & 1u) {}
};

// Wait (bounded) until what a ring of N was filled with in its last uses, of g in all, has arrived.
template <int N>
__device__ __forceinline__ void landed(uint64_t *full, uint32_t g) {
  for (uint32_t r = 1; r <= N && r <= g; ++r) {
    const Slot<N> s(g - r);
    if (!tc::mbar_wait_bounded(&full[s.at], s.parity, kDrain)) return;
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// a float of CTA r's copy of a shared variable
__device__ __forceinline__ float ld_cluster(const float *p, int r) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [ra];\n\t}\n"
      : "=f"(v)
      : "r"(tc::smem_u32(p)), "r"(r)
      : "memory");
  return v;
}
// Arrive on the pair's first CTA's copy of `bar`.  What the barrier orders is tensor memory (its
// own fences) and TMA's writes, no thread's stores, so no cluster-wide release is asked for: one
// (.release.cluster) held every arriving warp for hundreds of cycles, 531 -> 457 us for
// 16384 x 1536 x 6144 without it.
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}\n" ::"r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          tc::smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}
// untiled copy; both addresses and the size are multiples of 16 bytes
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n"
               "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::"r"(tc::smem_u32(dst))
               : "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(taddr) : "memory");
}
// B: MN-major, 128-byte swizzle, one atom (64 BF16) wide, 8-token groups 1024 bytes apart.  The
// descriptor's lower half holds the start address, the upper half is constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | ((uint32_t)(kBox >> 4) << 16); }
constexpr uint32_t kIdesc = tc::idesc_bf16(256, 128) | (1u << 16);   // B is MN-major
// D (+)= A[tmem] B[smem], one 256 x 128 x 16 step over both CTAs
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t bdesc_lo, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\t"
      "mov.b64 bd, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], bd, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(bdesc_lo), "n"(kDescHi), "n"(kIdesc), "r"(accumulate)
      : "memory");
}
// arrive on both CTAs' `bar` once the MMAs issued so far have completed
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
          tc::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// one thread of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok != 0;
}

__device__ __forceinline__ void ldmatrix_t8(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 x, y;
  *reinterpret_cast<uint32_t *>(&x) = a;
  *reinterpret_cast<uint32_t *>(&y) = b;
  x = __hmul2(x, y);
  return *reinterpret_cast<uint32_t *>(&x);
}
// Four codes c -> two BF16 pairs of code * 2^-120 (2^-112 for E5M2): the sign stays the top bit, the
// exponent and mantissa bits move to the BF16 fields, a code's subnormals become BF16's.  Done on
// all four at once (upper bytes, lower bytes), then interleaved.
template <int F>
__device__ __forceinline__ void spread_codes(uint32_t c, uint32_t &w0, uint32_t &w1) {
  constexpr int down = F == FMT_E4M3 ? 4 : 3;
  constexpr uint32_t top = F == FMT_E4M3 ? 0x07070707u : 0x0F0F0F0Fu, low = F == FMT_E4M3 ? 0xF0F0F0F0u : 0xE0E0E0E0u;
  const uint32_t hi = ((c >> down) & top) | (c & 0x80808080u), lo = (c << (8 - down)) & low;
  w0 = __byte_perm(lo, hi, 0x5140);
  w1 = __byte_perm(lo, hi, 0x7362);
}
template <int F, int NH, int TERMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_weight_grad(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap tm_codes,
                  const __grid_constant__ CUtensorMap tm_delta, int *status) {
  using C = Cfg<NH, TERMS>;
  static_assert(C::smem + sizeof(Shared<NH, TERMS>) <= 227 * 1024, "a CTA's shared memory");
  constexpr int kCodes = C::codes, kDeltas = C::deltas, kPeriod = C::period;
  extern __shared__ uint8_t dsm[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(((uintptr_t)dsm + 1023) & ~(uintptr_t)1023);
  uint8_t *const sm_delta = sm + kCodes * kBox;
  __shared__ Shared<NH, TERMS> sh;
  auto &cfull = sh.cfull, &cempty = sh.cempty;
  auto &bfull = sh.bfull, &bempty = sh.bempty;
  auto &dfull = sh.dfull, &dempty = sh.dempty;
  uint64_t *const ready = sh.ready;
  auto &scale_sh = sh.scales;
  volatile int &failed = sh.failed;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  grid_release();   // k_join_slices

  if (warp == 0) alloc_pair(&sh.tmem);
  if (tid == 32) {
    for (int s = 0; s < kCodes; ++s) {
      tc::mbar_init(&cfull[s], 1);
      tc::mbar_init(&cempty[s], 4);
    }
    for (int s = 0; s < kDeltas; ++s) {
      tc::mbar_init(&bfull[s], 1);
      tc::mbar_init(&bempty[s], NH);
    }
    for (int s = 0; s < kGroup; ++s) tc::mbar_init(&ready[s], 2 * 4);
    for (int b = 0; b < 3; ++b) {
      tc::mbar_init(&dfull[b], 1);
      tc::mbar_init(&dempty[b], 2 * kFoldWarps);
    }
    tc::mbar_init(&sh.drained, NH);
    tc::fence_mbar_init();
    failed = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  // Called by whole warps: the lanes go on together, or none does.  A try waits up to 4 us itself (to look first
  // and try then cost the 16384 x 1536 x 6144 product 1.5 %).
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    bool done = tc::mbar_try_wait(bar, parity);
    if (!done) {
      const long long t0 = clock64();
      do {
        if (failed || clock64() - t0 > P.budget) {
          failed = 1;
          set_status(status, GIFT_ERR_TIMEOUT);
          break;
        }
        done = tc::mbar_try_wait(bar, parity);
      } while (!done);
    }
    return __all_sync(0xFFFFFFFFu, done) != 0;
  };

  // registers: 72 per thread at launch (504 over the seven groups of four warps), redistributed as
  // 2 x 152 + 5 x 40
  if (warp < kDeqWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    // Each of these warps walks its loop whole, so that addresses and coordinates stay in uniform
    // registers, which TMA and the MMAs take; one elected thread issues.
    const bool one = elect_one();
    if (warp == kCodesWarp || warp == kDeltaWarp) {
      // ---------------- TMA ----------------
      uint32_t g = 0;   // stages so far
      bool ok = true;
      grid_wait();   // what the kernels before this one wrote is there
      if (warp == kCodesWarp) {
        for (int it = pair; it < P.items && ok; it += pairs) {
          const Item w(P, it, 128 * NH);
          // the CTA's columns are one group; past d_in the codes are ones for db, otherwise zeros
          const int i = w.i0 + 128 * rank;
          const bool ones = P.ones >= 0 && i >= P.ones;
          const StageScales *scales = P.scales + (size_t)min(i / kActGroup, P.last_group) * P.stages + w.t0 / kK;
          for (int t = w.t0; t < w.t0 + kGroup * kK * w.ng; t += kK, ++g, ++scales) {
            const Slot<kCodes> c(g);
            if (!(ok = wait(&cempty[c.at], c.parity ^ 1u))) break;
            if (one) {
              tc::mbar_arrive_expect_tx(&cfull[c.at], kBox + kScaleBytes);
              if (ones) bulk_load(sm + c.at * kBox, P.one_codes, kBox, &cfull[c.at]);
              else tc::tma_load_2d(sm + c.at * kBox, &tm_codes, i, t, &cfull[c.at]);
              bulk_load(&scale_sh[c.at], scales, kScaleBytes, &cfull[c.at]);
            }
          }
        }
        landed<kCodes>(cfull, g);
      } else {
        for (int it = pair; it < P.items && ok; it += pairs) {
          const Item w(P, it, 128 * NH);
          for (int t = w.t0; t < w.t0 + kGroup * kK * w.ng; t += kK, ++g) {
            const Slot<kDeltas> d(g);
            if (!(ok = wait(&bempty[d.at], d.parity ^ 1u))) break;
            if (one) {
              uint64_t *bar = &bfull[d.at];
              uint8_t *st = sm_delta + d.at * C::delta_bytes;
              tc::mbar_arrive_expect_tx(bar, C::delta_bytes);
#pragma unroll
              for (int b = 0; b < NH * TERMS; ++b)   // box b: half b / TERMS, term b % TERMS
                tma_load_3d(st + b * kBox, &tm_delta, w.o0 + 128 * (b / TERMS) + 64 * rank, t, b % TERMS, bar);
            }
          }
        }
        // leave no arrival of the MMAs' commits behind: the last stages'
        for (uint32_t r = 1; ok && r <= kDeltas && r <= g; ++r) {
          const Slot<kDeltas> d(g - r);
          ok = wait(&bempty[d.at], d.parity);
        }
        landed<kDeltas>(bfull, g);
        // the pair's first CTA may have a wait of its own to end before its last commit
        tc::mbar_wait_bounded(&sh.drained, 0, P.budget + kDrain);
      }
    } else if ((warp == kMmaWarp || (NH == 2 && warp == kMmaWarp + 2)) && rank == 0) {
      // ---------------- MMA, a warp per half of the tile: a warp's waits and commits cost about as
      // much as its half's MMAs, so two warps keep the queue full ----------------
      const uint32_t b_first = desc_lo(tc::smem_u32(sm_delta)), a0 = tmem + kACol;
      Accumulators<NH> acc;
      auto walk = [&](auto half_c) {
        constexpr int half = decltype(half_c)::value;
        uint32_t n = 0;
        for (int it = pair; it < P.items; it += pairs) {
          const int ng = Item(P, it, 128 * NH).ng;
          acc.start_tile();
          // both halves' changes of accumulator are followed and waited for: each phase is seen once
#pragma unroll
          for (int h = 0; h < NH; ++h)
            if (!wait(&dempty[acc.cur(h)], acc.use(acc.cur(h)) ^ 1u)) return;
          for (int gi = 0; gi < ng; ++gi, ++n) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
              constexpr int kHalf = kPeriod / 2;
              if (j % kPeriod == 0 && (j || gi)) {
                acc.next(0);
                if (!wait(&dempty[acc.cur(0)], acc.use(acc.cur(0)) ^ 1u)) return;
              }
              if (NH == 2 && j % kPeriod == kHalf) {
                acc.next(1);
                if (!wait(&dempty[acc.cur(1)], acc.use(acc.cur(1)) ^ 1u)) return;
              }
              const int mine = acc.cur(half);
              const bool fresh = j % kPeriod == half * kHalf || (half == 1 && j == 0 && gi == 0);
              const uint32_t db = (kGroup * n + j) % kDeltas;
              const uint32_t b0 = b_first + (db * NH + half) * TERMS * (kBox >> 4);
              if (!wait(&ready[j], n & 1u)) return;
              tc::fence_after_sync();
              if (one) {
#pragma unroll
                for (int k = 0; k < kK / 16; ++k)
#pragma unroll
                  for (int p = 0; p < TERMS; ++p)
                    mma_pair(tmem + 128 * mine, a0 + 32 * j + 8 * k,
                             b0 + p * (kBox >> 4) + 128 * k,
                             k == 0 && p == 0 ? (fresh ? 0u : 1u) : 1u);
                commit_pair(&bempty[db]);
                if ((j + 1) % kPeriod == half * kHalf || (half == 1 && j + 1 == kGroup && gi + 1 == ng))
                  commit_pair(&dfull[mine]);
              }
            }
          }
        }
      };
      if (warp == kMmaWarp) walk(std::integral_constant<int, 0>());
      else walk(std::integral_constant<int, 1>());
      if (one) commit_pair(&sh.drained);
    }
  } else if (warp < kFoldWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    // ---------------- codes -> BF16 in tensor memory: 32 of the CTA's rows i of every fourth stage ----------------
    const int dw = warp - kDeqWarp, q = dw & 3, turn = dw >> 2;
    uint32_t total = 0;
    for (int it = pair; it < P.items; it += pairs) total += (uint32_t)Item(P, it, 128 * NH).ng;
    const uint32_t mine = tc::smem_u32(sm) + lane * 128, slot = tmem + kACol + 32 * turn + ((uint32_t)(32 * q) << 16);
    for (uint32_t n = 0; n < total; ++n) {
      const uint32_t g = kGroup * n + turn;
      const Slot<kCodes> c(g);
      const Slot<kDeltas> d(g);
      if (!wait(&cfull[c.at], c.parity)) break;
      const StageScales &sc = scale_sh[c.at];
      bool ok = true;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t v[8], x[16];
        const uint32_t from = mine + c.at * kBox + (((2 * q + hh) ^ (lane & 7)) << 4);
        ldmatrix_t8(from, v);
        ldmatrix_t8(from + 32 * 128, v + 4);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint2 s = *reinterpret_cast<const uint2 *>(&sc.first[16 * m + 4 * (lane & 3)]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t w0, w1;
            spread_codes<F>(v[2 * m + u], w0, w1);
            x[4 * m + 2 * u] = mul_bf16x2(w0, s.x);
            x[4 * m + 2 * u + 1] = mul_bf16x2(w1, s.y);
          }
        }
        if (sc.any_over) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t o = *reinterpret_cast<const uint32_t *>(&sc.over[16 * m + 4 * (lane & 3)]);
            const uint32_t sx = 0x3F803F80u + ((o & 0xFFu) << 7) + ((o & 0xFF00u) << 15),
                           sy = 0x3F803F80u + ((o >> 9) & 0x7F80u) + ((o >> 24) << 23);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[4 * m + u] = mul_bf16x2(x[4 * m + u], u & 1 ? sy : sx);
          }
        }
        if (hh == 0) {
          // The slot's last MMAs, a group ago, are done: their delta is free (its barrier cannot be a phase
          // further yet), or, with one group of stages, this one's delta has been loaded in its place.
          if (kDeltas > kGroup) {
            if (n > 0) {
              const Slot<kDeltas> before(g - kGroup);
              ok = wait(&bempty[before.at], before.parity);
            }
          } else {
            ok = wait(&bfull[d.at], d.parity);
          }
          if (!ok) break;
          tc::fence_after_sync();
        }
        tmem_st_16x256b_x4(slot + ((uint32_t)(16 * hh) << 16), x);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&cempty[c.at]);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      // one of the stage's warps answers for this CTA's half of delta
      if (kDeltas > kGroup && q == 0 && !wait(&bfull[d.at], d.parity)) break;
      __syncwarp();
      if (lane == 0) arrive_first(&ready[turn]);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;\n");
    // ---------------- fold and store (this warp: 32 rows i, 64 of each half's columns) ----------------
    const int q = warp & 3, c = (warp - kFoldWarp) >> 2;
    const uint32_t off = ((uint32_t)(32 * q) << 16) + 64 * c;
    Accumulators<NH> acc;
    bool ok = true;
    for (int it = pair; it < P.items && ok; it += pairs) {
      const Item w(P, it, 128 * NH);
      float2 sum[NH][32];
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 32; ++e) sum[h][e] = make_float2(0.0f, 0.0f);
      // add half h's finished segment and hand its accumulator back
      auto fold = [&](int h, float2(&to)[32]) {
        const int b = acc.cur(h);
        if (!(ok = ok && wait(&dfull[b], acc.use(b)))) return;
        tc::fence_after_sync();
#pragma unroll
        for (int e = 0; e < 64; e += 16) {
          uint32_t raw[16];
          tc::tmem_ld16_nowait(tmem + off + 128 * b + e, raw);
          tc::tmem_wait_ld16(raw);
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            float2 &s = to[(e + x) / 2];
            s = add2(s, make_float2(__uint_as_float(raw[x]), __uint_as_float(raw[x + 1])));
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_first(&dempty[b]);
      };
      acc.start_tile();
#pragma unroll 1
      for (int seg = 1; seg <= w.ng * (kGroup / kPeriod) && ok; ++seg) {
        if (NH == 2) {   // half 1 changes in the middle of half 0's segment, and at the end
          fold(1, sum[NH - 1]);
          acc.next(1);
        }
        fold(0, sum[0]);
        if (seg < w.ng * (kGroup / kPeriod)) acc.next(0);
      }
      if (NH == 2) fold(1, sum[NH - 1]);
      if (!ok) break;
      const int i = w.i0 + 128 * rank + 32 * q + lane;
      auto store = [&](float *p, size_t step, float ga) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const int o = w.o0 + 128 * h + 64 * c;
          float *r = p + o * step;
#pragma unroll
          for (int e = 0; e < 64; ++e, r += step) {
            if (o + e >= P.d_out) break;
            *r = (e & 1 ? sum[h][e / 2].y : sum[h][e / 2].x) * ga;
          }
        }
      };
      if (i < P.d_in) store(P.out + (size_t)w.slice * P.d_out * P.d_in + i, P.d_in, P.gamma ? P.gamma[i] : 1.0f);
      else if (i == P.ones) store(P.db + (size_t)w.slice * P.d_out, 1, 1.0f);
    }
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

// ---- few outputs: FP32 SIMT in one launch ----------------------------------------------------------
// 32 x 32 tiles of dW, a cluster of eight CTAs each: a CTA takes every eighth 64 tokens through shared
// memory, eight of them per warp, each lane 4 x 8 outputs in packed FP32.  A warp's sums are folded
// every 64 tokens of the batch, the eight warps' joined in order, then the eight CTAs' through
// distributed shared memory; db alongside.  Bound by latency: 512 x 64 x 256 takes about 6 us.
constexpr int kSmallTokens = 2048;   // see small_product
constexpr int kSmTok = 64, kSmTile = 32, kSmThreads = 256, kSmCtas = 8;

template <int F, typename E>
__global__ void __cluster_dims__(kSmCtas, 1, 1) __launch_bounds__(kSmThreads, 1)
    k_weight_grad_small(const E *__restrict__ delta, const uint8_t *__restrict__ codes,
                        const uint8_t *__restrict__ scales, int T, int d_out, int d_in, int groups,
                        const float *__restrict__ gamma, const float *__restrict__ beta, float *__restrict__ db_out,
                        float *__restrict__ dW) {
  __shared__ __align__(16) union {
    struct {
      float delta[kSmTok][kSmTile], v[kSmTok][kSmTile];
    } in;
    float out[8][kSmTile][kSmTile + 1];
  } sh;
  __shared__ float sh_db[8][kSmTile];
  __shared__ float cta[kSmTile][kSmTile + 1];   // the CTA's sums; column 32: db
  const int rank = (int)cluster_rank();
  const int i0 = blockIdx.x / kSmCtas * kSmTile, o0 = blockIdx.y * kSmTile;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, lo = 4 * (lane >> 2), li = 8 * (lane & 3);
  const bool o_in = o0 + lane < d_out, i_in = i0 + lane < d_in;
  const E *dp = delta + o0 + lane;
  const uint8_t *cp = codes + i0 + lane, *sp = scales + i0 / kActGroup;   // a tile lies in one group
  float2 tot[4][4];
  float db = 0.0f;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) tot[a][b] = make_float2(0.0f, 0.0f);
  constexpr int kPer = kSmTok / 8;
  float rd[kPer];
  uint32_t rc[kPer], rs[kPer];
  auto load = [&](int t0) {   // token t0 + w + 8 k of the chunk, this lane's column
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int t = t0 + w + 8 * k;
      rd[k] = t < T && o_in ? ld1(dp + (size_t)t * d_out) : 0.0f;
      rc[k] = t < T && i_in ? cp[(size_t)t * d_in] : 0u;
      rs[k] = t < T ? sp[(size_t)t * groups] : 127u;
    }
  };
  load(rank * kSmTok);
  for (int t0 = rank * kSmTok; t0 < T; t0 += kSmTok * kSmCtas) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      sh.in.delta[w + 8 * k][lane] = rd[k];
      sh.in.v[w + 8 * k][lane] = dec_fp8<F>(rc[k]) * act_scale(rs[k]);
    }
    __syncthreads();
    load(t0 + kSmTok * kSmCtas);
    float2 acc[4][4];
    float dsum = 0.0f;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < kPer; ++k) {
      const int r = kPer * w + k;
      const float4 d4 = *reinterpret_cast<const float4 *>(&sh.in.delta[r][lo]);
      const float4 va = *reinterpret_cast<const float4 *>(&sh.in.v[r][li]),
                   vb = *reinterpret_cast<const float4 *>(&sh.in.v[r][li + 4]);
      const float2 v[4] = {make_float2(va.x, va.y), make_float2(va.z, va.w), make_float2(vb.x, vb.y),
                           make_float2(vb.z, vb.w)};
      const float d[4] = {d4.x, d4.y, d4.z, d4.w};
      dsum += sh.in.delta[r][lane];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fma2(both(d[a]), v[b], acc[a][b]);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) tot[a][b] = add2(tot[a][b], acc[a][b]);
    db += dsum;
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      sh.out[w][lo + a][li + 2 * b] = tot[a][b].x;
      sh.out[w][lo + a][li + 2 * b + 1] = tot[a][b].y;
    }
  sh_db[w][lane] = db;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int o = w + 8 * k;
    float v = sh.out[0][o][lane], b = sh_db[0][o];
#pragma unroll
    for (int x = 1; x < 8; ++x) {
      v += sh.out[x][o][lane];
      b += sh_db[x][o];
    }
    cta[o][lane] = v;
    if (lane == 0) cta[o][kSmTile] = b;
  }
  cluster_sync();
  // rows 4 rank .. 4 rank + 3 of the tile are joined and stored by this CTA, a warp each
  if (w < 4) {
    const int o = 4 * rank + w;
    float v = 0.0f, b = 0.0f;
#pragma unroll
    for (int r = 0; r < kSmCtas; ++r) {
      v += ld_cluster(&cta[o][lane], r);
      b += ld_cluster(&cta[o][kSmTile], r);
    }
    if (o0 + o < d_out) {
      if (db_out && i0 == 0 && lane == 0) db_out[o0 + o] = b;
      if (i_in) {
        if (gamma) v *= gamma[i0 + lane];
        if (beta) v = fmaf(beta[i0 + lane], b, v);
        dW[(size_t)(o0 + o) * d_in + i0 + lane] = v;
      }
    }
  }
  cluster_sync();   // no CTA leaves while another reads its sums
}

// dW = gamma * (the slices' sums in order) + beta db; db likewise from its slices.  `part` may be dW
// (one slice).  A CTA takes 2048 columns of every gridDim.y-th row; eight loads a thread are in flight.
// Bound by L2 where that holds the sums: gain and offset onto 1536 x 6144 outputs take 16 us more
// (75 MB, 4.7 TB/s), onto 1021 x 2731 5 us.
constexpr int kJoinCols = 8;   // per thread
__global__ void __launch_bounds__(256) k_join_slices(const float *part, int slices, int d_out, int d_in,
                                                     const float *gamma, const float *beta, const float *db_part,
                                                     int db_slices, float *db, float *dW) {
  grid_wait();
  const size_t n = (size_t)d_out * d_in;
  const int c0 = blockIdx.x * 256 * kJoinCols + threadIdx.x;
  float ga[kJoinCols], be[kJoinCols];
#pragma unroll
  for (int k = 0; k < kJoinCols; ++k) {
    const int i = c0 + 256 * k;
    ga[k] = gamma && i < d_in ? gamma[i] : 1.0f;
    be[k] = beta && i < d_in ? beta[i] : 0.0f;
  }
  for (int o = blockIdx.y; o < d_out; o += gridDim.y) {
    const size_t row = (size_t)o * d_in;
    float v[kJoinCols], b = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinCols; ++k) v[k] = c0 + 256 * k < d_in ? part[row + c0 + 256 * k] : 0.0f;
    if (db_part) b = db_part[o];
    for (int s = 1; s < slices; ++s) {
#pragma unroll
      for (int k = 0; k < kJoinCols; ++k)
        if (c0 + 256 * k < d_in) v[k] += part[s * n + row + c0 + 256 * k];
      if (s < db_slices) b += db_part[(size_t)s * d_out + o];
    }
    if (db && c0 == 0) db[o] = b;
#pragma unroll
    for (int k = 0; k < kJoinCols; ++k)
      if (c0 + 256 * k < d_in) dW[row + c0 + 256 * k] = beta ? fmaf(be[k], b, v[k] * ga[k]) : v[k] * ga[k];
  }
}

// ---- what the tensor-core kernel reads, made by one launch -------------------------------------------
// Independent parts share the launch, each on its own CTAs: scales by group and stage (16384 x 6144: 5 us
// cold), copies with aligned rows (5003 x 1021 BF16 and 5003 x 2731 codes: 42 us a call with them, 37
// without), FP32 delta's terms, delta's sums over tokens (16384 x 1536 BF16: 16 us).  Bound by HBM and
// by the launch; the product's launch overlaps its end (griddepcontrol).
struct Prepare {
  const uint8_t *scales;       // [T][groups]
  StageScales *stage_scales;   // [rows][stages]
  uint8_t *one_codes;          // a box of the code of 1
  int T, groups, stages;
  int rows;                    // groups, or one more: the group of ones
  int nscale, nsums, ndelta, ncodes;   // CTAs of each part, in this order
  int sum_slices, sum_rows;    // nsums > 0: sums of delta over slices of consecutive tokens
  bool sum_vec;
  float *sum_part;             // [sum_slices][d_out]
  const void *delta;           // ndelta > 0: FP32 -> three BF16 terms, or BF16 rows of another pitch
  void *delta_out;
  int d_out, delta_ld;         // delta_ld: elements
  const uint8_t *codes;        // ncodes > 0: rows of another pitch
  uint8_t *codes_out;
  int d_in;
  size_t codes_ld;
};

// Scale bytes -> StageScales (NaN for a marked group, 1 past T and for ones): a stage of 64 tokens x 64 groups per CTA
// through shared memory, a warp writes a group.
template <int F>
__device__ __forceinline__ void stage_scales(const Prepare &P, int cta, uint8_t (*tile)[65]) {
  constexpr int up = F == FMT_E4M3 ? 120 : 112;
  const int stage = cta % P.stages, g0 = cta / P.stages * 64, ng = min(64, P.rows - g0), t0 = stage * kK;
  const int lane = threadIdx.x & 31;
  uint8_t b[kK / 8][2];   // all loads before the first store
#pragma unroll
  for (int k = 0; k < kK / 8; ++k)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + (threadIdx.x >> 5) + 8 * k, g = g0 + lane + 32 * u;
      b[k][u] = t < P.T && g < P.groups ? P.scales[(size_t)t * P.groups + g] : 127;
    }
#pragma unroll
  for (int k = 0; k < kK / 8; ++k)
#pragma unroll
    for (int u = 0; u < 2; ++u) tile[(threadIdx.x >> 5) + 8 * k][lane + 32 * u] = b[k][u];
  __syncthreads();
  for (int c = threadIdx.x >> 5; c < ng; c += 8) {
    uint32_t first[2], over[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int b = tile[2 * lane + u][c];
      over[u] = b == (int)kActBad ? 0u : (uint32_t)max(0, b + up - 254);
      first[u] = b == (int)kActBad ? 0x7FC0u : (uint32_t)(b + up - (int)over[u]) << 7;
    }
    StageScales &o = P.stage_scales[(size_t)(g0 + c) * P.stages + stage];
    reinterpret_cast<uint32_t *>(o.first)[lane] = first[0] | first[1] << 16;
    reinterpret_cast<uint16_t *>(o.over)[lane] = (uint16_t)(over[0] | over[1] << 8);
    const bool any = __any_sync(0xFFFFFFFFu, (over[0] | over[1]) != 0);
    if (lane == 0) o.any_over = any;
  }
}

// Sums over a slice of tokens of one piece of 512 columns: a warp takes every eighth token, the eight
// warps' sums are joined in order.
template <typename E, bool VEC>
__device__ __forceinline__ void column_sums(const Prepare &P, int cta, float (*sh)[16 * 33]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c0 = cta / P.sum_slices * kPiece, slice = cta % P.sum_slices, n = P.d_out - c0;
  const int t1 = min(P.T, (slice + 1) * P.sum_rows);
  float2 s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = both(0.0f);
#pragma unroll 4
  for (int t = slice * P.sum_rows + w; t < t1; t += 8) {
    Raw<E> r;
    load_piece<VEC>(static_cast<const E *>(P.delta) + (size_t)t * P.d_out + c0, n, lane, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = add2(s[k], r.pair(k));
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) sh[w][33 * e + lane] = e & 1 ? s[e / 2].y : s[e / 2].x;
  __syncthreads();
  for (int c = threadIdx.x; c < kPiece && c < n; c += 256) {
    const int at = VEC ? 33 * (c % 16) + c / 16 : 33 * (c / 32) + c % 32;
    float v = sh[0][at];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += sh[k][at];
    P.sum_part[(size_t)slice * P.d_out + c0 + c] = v;
  }
}

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

// FP32 as three BF16 terms (exact from 2^-110 up; below, the last ends at BF16's smallest step), planes of
// T rows of ld columns; a warp per row, two columns per lane
__device__ __forceinline__ void bf16_terms(const float *x, int T, int d, int ld, uint16_t *out, int cta, int ctas) {
  const size_t plane = (size_t)T * ld;
  for (int t = cta * 8 + (threadIdx.x >> 5); t < T; t += ctas * 8) {
    const float *p = x + (size_t)t * d;
    uint16_t *o = out + (size_t)t * ld;
    for (int c = 2 * (threadIdx.x & 31); c < d; c += 64) {   // ld is even
      uint32_t w[3];
      const float x0 = p[c], x1 = c + 1 < d ? p[c + 1] : 0.0f;
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
      for (int k = 0; k < 3; ++k) *reinterpret_cast<uint32_t *>(o + k * plane + c) = w[k];
    }
  }
}

// Rows of `bytes` bytes at any alignment -> rows of ld (a multiple of 16) bytes; a warp per row, 16 bytes
// per lane from the two aligned blocks that hold them.  Past a row's end nothing is read again (the
// tensor map's width).
__device__ __forceinline__ uint4 aligned_block(uintptr_t p, uintptr_t lo, uintptr_t hi) {
  if (p >= lo && p + 16 <= hi) return *reinterpret_cast<const uint4 *>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};   // the ends of the matrix
#pragma unroll
  for (int b = 0; b < 16; ++b)
    if (p + b >= lo && p + b < hi) w[b / 4] |= (uint32_t)*reinterpret_cast<const uint8_t *>(p + b) << (8 * (b % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void repitch(const uint8_t *src, int T, size_t bytes, size_t ld, uint8_t *dst, int cta,
                                        int ctas) {
  const uintptr_t lo = (uintptr_t)src, hi = lo + (size_t)T * bytes;
  for (int t = cta * 8 + (threadIdx.x >> 5); t < T; t += ctas * 8) {
    const uintptr_t row = lo + (size_t)t * bytes;
    const int off = (int)(row & 15), sh = 8 * (off & 3);
#pragma unroll 4
    for (size_t c = 16 * (threadIdx.x & 31); c < bytes; c += 512) {
      const uintptr_t at = row + c - off;
      const uint4 a = aligned_block(at, lo, hi), b = off ? aligned_block(at + 16, lo, hi) : a;
      uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (off & 8) {   // the same for the whole row
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
      }
      if (off & 4) {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
      }
      *reinterpret_cast<uint4 *>(dst + t * ld + c) =
          make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                     __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
    }
  }
}

template <int F, bool BF16>
__global__ void __launch_bounds__(256) k_prepare(const __grid_constant__ Prepare P) {
  __shared__ union {
    uint8_t tile[kK][65];
    float sums[8][16 * 33];   // a lane's 16 columns 33 words apart: neither side conflicts
  } sh;
  grid_release();
  int cta = blockIdx.x;
  if (cta < P.nscale) {
    constexpr uint32_t one = F == FMT_E4M3 ? 0x38383838u : 0x3C3C3C3Cu;
    if (cta == 0)
      for (int e = threadIdx.x; e < kBox / 16; e += 256)
        reinterpret_cast<uint4 *>(P.one_codes)[e] = make_uint4(one, one, one, one);
    stage_scales<F>(P, cta, sh.tile);
    return;
  }
  cta -= P.nscale;
  if (cta < P.nsums) {
    using E = typename std::conditional<BF16, __nv_bfloat16, float>::type;
    if (P.sum_vec) column_sums<E, true>(P, cta, sh.sums);
    else column_sums<E, false>(P, cta, sh.sums);
    return;
  }
  cta -= P.nsums;
  if (cta < P.ndelta) {
    if (BF16)
      repitch(static_cast<const uint8_t *>(P.delta), P.T, (size_t)P.d_out * 2, (size_t)P.delta_ld * 2,
              static_cast<uint8_t *>(P.delta_out), cta, P.ndelta);
    else
      bf16_terms(static_cast<const float *>(P.delta), P.T, P.d_out, P.delta_ld, static_cast<uint16_t *>(P.delta_out),
                 cta, P.ndelta);
    return;
  }
  repitch(P.codes, P.T, P.d_in, P.codes_ld, P.codes_out, cta - P.ndelta, P.ncodes);
}

// ---- host ---------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// `planes` matrices of rows x cols elements, rows `pitch` bytes apart, read in 128-byte x 64-row boxes
bool boxes(CUtensorMap *m, bool bf16, const void *base, int rows, int cols, size_t pitch, int planes) {
  const auto enc = encoder();
  if (!enc) return false;
  const int rank = bf16 ? 3 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {pitch, pitch * (cuuint64_t)rows};
  const cuuint32_t box[3] = {bf16 ? 64u : 128u, (cuuint32_t)kK, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
             const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t pad16(size_t bytes) { return (bytes + 15) / 16 * 16; }

struct Plan {
  int nh, mt, nt, ng, slices, pairs;
  bool ones;
  double cost;   // in the time of a group, 1.1 us at 256 columns
};

// Tiles of 256 x 256, or 256 x 128 where one half covers d_out; with `ones`, the columns' groups are
// followed by one of ones, whose sums are db.  Tokens are cut into slices where the tiles alone leave
// pairs of SMs idle: the count with the least waves x (groups of an item + its start and end, about 1
// group) + the slices' own traffic (written and read once, about 4 MB in the time of a group; the join
// kernel's launch about 2 groups).
Plan plan_of(int sms, int T, int d_out, int d_in, bool ones) {
  Plan p;
  p.nh = d_out <= 128 ? 1 : 2;
  p.mt = ((d_in + kActGroup - 1) / kActGroup + ones + 1) / 2;
  p.nt = (d_out + 128 * p.nh - 1) / (128 * p.nh);
  p.ng = (T + kGroup * kK - 1) / (kGroup * kK);
  p.pairs = sms / 2 > 1 ? sms / 2 : 1;
  const long long tiles = (long long)p.mt * p.nt;
  const double traffic = 8.0 * d_out * d_in / 4.0e6;
  p.ones = ones;
  p.slices = 1;
  p.cost = 1e300;
  for (int s = 1; s <= 64 && s <= p.ng; ++s) {
    const long long waves = (tiles * s + p.pairs - 1) / p.pairs;
    const double cost = (double)waves * ((p.ng + s - 1) / s + 1) + (s > 1 ? 2.0 + s * traffic : 0.0);
    if (cost < p.cost) {
      p.cost = cost;
      p.slices = s;
    }
  }
  return p;
}

// With db: from the group of ones, which is free where the last tile has room for it (5003 x 1021 x 2731
// BF16: 54 us, by a pass over delta 63) or there is an idle pair of SMs in the last wave (16384 x 1536 x
// 6144: 194 us, 193 without db, 204 by the pass; FP32 521 and 534), or by the pass over delta, about 5
// MB in the time of a group and 4 groups for its second kernel, where the tiles of ones would take a
// wave more (16384 x 6144 x 1536: 271 us with them, 234 by the pass, 192 without db).  Single calls,
// caches flushed between them.
Plan plan_for(int sms, bool bf16, int T, int d_out, int d_in, bool need_db) {
  const Plan p = plan_of(sms, T, d_out, d_in, false);
  if (!need_db) return p;
  const Plan ones = plan_of(sms, T, d_out, d_in, true);
  return ones.cost <= p.cost + 4.0 + (double)T * d_out * (bf16 ? 2 : 4) / 5.0e6 ? ones : p;
}

// Slices of tokens for delta's sums: about four CTAs per SM with all pieces, 64 tokens at least.
int sum_slices(int sms, int T, int d_out) {
  const int pieces = (d_out + kPiece - 1) / kPiece, most = (T + 63) / 64;
  const int s = (4 * sms + pieces - 1) / pieces;
  return s < most ? s : most;
}

template <int F, int NH, int TERMS>
cudaError_t launch(const Launch &L, const Params &P, const CUtensorMap &tc_, const CUtensorMap &td, int pairs) {
  using C = Cfg<NH, TERMS>;
  const cudaError_t e = ensure_dynamic_smem<k_weight_grad<F, NH, TERMS>>(C::smem);
  if (e != cudaSuccess) return e;
  // launched while k_prepare still runs (grid_wait)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (P.items < pairs ? P.items : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = L.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_weight_grad<F, NH, TERMS>, P, tc_, td, L.status);
}

template <int F>
cudaError_t launch_fmt(const Launch &L, const Params &P, const CUtensorMap &tc_, const CUtensorMap &td, const Plan &p,
                       bool bf16) {
  if (bf16) return p.nh == 1 ? launch<F, 1, 1>(L, P, tc_, td, p.pairs) : launch<F, 2, 1>(L, P, tc_, td, p.pairs);
  return p.nh == 1 ? launch<F, 1, 3>(L, P, tc_, td, p.pairs) : launch<F, 2, 3>(L, P, tc_, td, p.pairs);
}

// CTAs of eight warps, a row each, up to eight per SM
int row_grid(const Launch &L, int T) {
  const int c = (T + 7) / 8;
  return c < L.sms * 8 ? c : L.sms * 8;
}

}  // namespace

WeightGradWs weight_grad_layout(int sms, bool bf16, int T, int d_out, int d_in) {
  WeightGradWs w;
  const Plan p = plan_for(sms, bf16, T, d_out, d_in, false), with_db = plan_for(sms, bf16, T, d_out, d_in, true);
  const int slices = p.slices > with_db.slices ? p.slices : with_db.slices;
  w.part_floats = with_db.ones ? 0 : (size_t)sum_slices(sms, T, d_out) * d_out;
  w.db_floats = (size_t)with_db.slices * d_out;
  w.slice_floats = slices > 1 ? (size_t)slices * d_out * d_in : 0;
  // a BF16 delta and the codes are copied only when their rows are not 16-byte aligned, which the
  // caller's pointers decide: room for both
  w.delta_bytes = (size_t)T * pad16((size_t)d_out * 2) * (bf16 ? 1 : 3);
  w.code_bytes = (size_t)T * pad16(d_in);
  w.scale_bytes = (size_t)p.ng * kGroup * kScaleBytes * ((d_in + kActGroup - 1) / kActGroup + 1) + kBox;
  return w;
}

// Where the tensor-core kernel's fixed cost (its first loads, and the kernels before it) outweighs the
// small kernel's, whose clusters all run at once over a few chunks each.  A call with db: 512 x 64 x 256
// FP32 10.4 us here, 17.8 there; 2048 x 64 x 256 BF16 16.6 and 20.7; 4096 x 64 x 256 24.8 and 20.5.
bool small_product(int sms, int T, int d_out, int d_in) {
  const long long tiles = (long long)((d_out + kSmTile - 1) / kSmTile) * ((d_in + kSmTile - 1) / kSmTile);
  return tiles * kSmCtas <= 2 * sms && T <= kSmallTokens;
}

template <int F, typename E>
cudaError_t launch_small(const Launch &L, const WeightGrad &a) {
  const dim3 grid((a.d_in + kSmTile - 1) / kSmTile * kSmCtas, (a.d_out + kSmTile - 1) / kSmTile);
  k_weight_grad_small<F, E><<<grid, kSmThreads, 0, L.stream>>>(static_cast<const E *>(a.delta), a.codes, a.scales, a.T,
                                                               a.d_out, a.d_in, (a.d_in + kActGroup - 1) / kActGroup,
                                                               a.gamma, a.beta, a.db, a.dW);
  return cudaGetLastError();
}

cudaError_t launch_weight_grad(const Launch &L, int fmt, bool bf16, const WeightGrad &a) {
  if (small_product(L.sms, a.T, a.d_out, a.d_in)) {
    if (fmt == FMT_E4M3)
      return bf16 ? launch_small<FMT_E4M3, __nv_bfloat16>(L, a) : launch_small<FMT_E4M3, float>(L, a);
    return bf16 ? launch_small<FMT_E5M2, __nv_bfloat16>(L, a) : launch_small<FMT_E5M2, float>(L, a);
  }
  const bool need_db = a.db || a.beta;
  const Plan p = plan_for(L.sms, bf16, a.T, a.d_out, a.d_in, need_db);
  const bool join = p.slices > 1 || a.beta;
  // operands with 16-byte aligned rows, and the scales by group and stage
  Prepare q{};
  q.scales = a.scales;
  q.stage_scales = static_cast<StageScales *>(a.scale_ws);
  q.T = a.T;
  q.groups = (a.d_in + kActGroup - 1) / kActGroup;
  q.stages = p.ng * kGroup;
  q.rows = q.groups + p.ones;
  q.one_codes = reinterpret_cast<uint8_t *>(q.stage_scales + (size_t)q.stages * q.rows);
  q.nscale = q.stages * ((q.rows + 63) / 64);
  q.delta = a.delta;
  q.delta_out = a.delta_ws;
  q.d_out = a.d_out;
  q.codes = a.codes;
  q.codes_out = a.code_ws;
  q.d_in = a.d_in;
  if (need_db && !p.ones) {
    q.sum_slices = sum_slices(L.sms, a.T, a.d_out);
    q.sum_rows = (a.T + q.sum_slices - 1) / q.sum_slices;
    q.sum_vec = rows_vec(a.d_out, a.delta, nullptr);
    q.sum_part = a.part;
    q.nsums = q.sum_slices * ((a.d_out + kPiece - 1) / kPiece);
  }
  const void *delta = a.delta;
  size_t dpitch = (size_t)a.d_out * 2;
  if (!bf16 || dpitch % 16 || !aligned16(delta)) {
    dpitch = pad16(dpitch);
    q.delta_ld = (int)(dpitch / 2);
    q.ndelta = row_grid(L, a.T);
    delta = a.delta_ws;
  }
  const uint8_t *codes = a.codes;
  size_t cpitch = a.d_in;
  if (cpitch % 16 || !aligned16(codes)) {
    cpitch = q.codes_ld = pad16(cpitch);
    q.ncodes = row_grid(L, a.T);
    codes = a.code_ws;
  }
  const int pgrid = q.nscale + q.nsums + q.ndelta + q.ncodes;
  if (fmt == FMT_E4M3) {
    if (bf16) k_prepare<FMT_E4M3, true><<<pgrid, 256, 0, L.stream>>>(q);
    else k_prepare<FMT_E4M3, false><<<pgrid, 256, 0, L.stream>>>(q);
  } else {
    if (bf16) k_prepare<FMT_E5M2, true><<<pgrid, 256, 0, L.stream>>>(q);
    else k_prepare<FMT_E5M2, false><<<pgrid, 256, 0, L.stream>>>(q);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // db in slices where the product makes it in slices
  const int db_slices = p.ones ? p.slices : 1;
  float *const db = db_slices > 1 || !a.db ? a.db_ws : a.db;
  if (q.nsums && (e = launch_sum_parts(L, a.part, q.sum_slices, a.d_out, db)) != cudaSuccess) return e;

  CUtensorMap tm_codes, tm_delta;
  if (!boxes(&tm_codes, false, codes, a.T, a.d_in, cpitch, 1) ||
      !boxes(&tm_delta, true, delta, a.T, a.d_out, dpitch, bf16 ? 1 : 3))
    return cudaErrorInvalidValue;
  Params P;
  P.T = a.T;
  P.d_out = a.d_out;
  P.d_in = a.d_in;
  P.last_group = q.rows - 1;
  P.ng = p.ng;
  P.mt = p.mt;
  P.nt = p.nt;
  P.slices = p.slices;
  P.items = p.mt * p.nt * p.slices;
  P.scales = q.stage_scales;
  P.stages = q.stages;
  P.gamma = join ? nullptr : a.gamma;
  P.out = p.slices > 1 ? a.slices : a.dW;
  P.budget = L.barrier_wait;
  P.ones = p.ones ? q.groups * kActGroup : -1;
  P.one_codes = q.one_codes;
  P.db = db;
  e = fmt == FMT_E4M3 ? launch_fmt<FMT_E4M3>(L, P, tm_codes, tm_delta, p, bf16)
                      : launch_fmt<FMT_E5M2>(L, P, tm_codes, tm_delta, p, bf16);
  if (e != cudaSuccess || !join) return e;
  const int wide = (a.d_in + 256 * kJoinCols - 1) / (256 * kJoinCols), rows = (L.sms * 8 + wide - 1) / wide;
  return launch_after(L.stream, k_join_slices, dim3(wide, a.d_out < rows ? a.d_out : rows), 256, P.out, p.slices,
                      a.d_out, a.d_in, a.gamma, a.beta, need_db ? db : nullptr, db_slices, db_slices > 1 ? a.db : nullptr,
                      a.dW);
}

}  // namespace gift
