// What the tensor-core kernels that run on pairs of CTAs (a cluster of two SMs, cta_group::2) share:
// the pair's barriers, tensor memory and commits, rings of shared-memory slots, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "tc.cuh"

namespace gift {

constexpr long long kDrain = 4000000000LL;   // clocks that a leaving warp waits for what is in flight, about 2 s

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
__device__ __forceinline__ void alloc_pair(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n"
               "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::"r"(tc::smem_u32(dst))
               : "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(taddr) : "memory");
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

// ---- host ---------------------------------------------------------------------------------------
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

// `planes` matrices of rows x cols elements (one of bytes; BF16 any number), rows `pitch` bytes apart, read in boxes of
// 128 bytes x box_rows
inline bool boxes(CUtensorMap *m, bool bf16, const void *base, int rows, int cols, size_t pitch, int planes,
                  int box_rows) {
  const auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {pitch, pitch * (cuuint64_t)rows};
  const cuuint32_t box[3] = {bf16 ? 64u : 128u, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, bf16 ? 3 : 2,
             const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gift
