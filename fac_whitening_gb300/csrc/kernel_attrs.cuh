// What the host keeps per kernel and device between launches.  Host code only.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace gift {

constexpr int kKnownDevices = 64;

// Raises a kernel's opt-in dynamic shared-memory size to `bytes` where it is smaller, once per device and
// kernel for a fixed size (so no attribute call happens inside a stream capture after the first eager
// call).  The runtime's call sets the limit, down as well as up, so one thread at a time compares, calls and
// records: the limit never falls below what a launch has asked for.  Keyed on the kernel itself:
// instantiations that share a function type keep separate flags.
template <auto Kernel>
cudaError_t ensure_dynamic_smem(int bytes) {
  static std::atomic<int> done[kKnownDevices] = {};
  static std::mutex changing;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kKnownDevices;
  if (known && done[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  const std::lock_guard<std::mutex> one(changing);
  if (known && done[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void *>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) done[dev].store(bytes, std::memory_order_release);
  return e;
}

// CTAs of a kernel that an SM holds (at least 1), looked up once per device, CTA size and shared memory: a
// launch's grid, and with it the order of its sums, depends on that launch alone and not on the calls
// before it.  An entry is one word, written once; where two threads look up the same, both write the same.
template <auto Kernel>
int resident_per_sm(int threads, int smem) {
  constexpr int kEntries = 64;
  static std::atomic<unsigned long long> known[kEntries] = {};   // key and, in the low byte, the count; 0: free
  int dev = 0, per_sm = 0;
  const bool keep = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kKnownDevices;
  const unsigned long long key =
      (unsigned long long)smem << 32 | (unsigned long long)(threads / 32) << 16 | (unsigned long long)(dev & 63) << 8;
  int at = 0;
  for (; keep && at < kEntries; ++at) {
    const unsigned long long k = known[at].load(std::memory_order_relaxed);
    if (k == 0) break;
    if ((k & ~0xFFull) == key) return (int)(k & 0xFF);
  }
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, reinterpret_cast<const void *>(Kernel), threads, smem) !=
          cudaSuccess || per_sm < 1)
    return 1;
  for (; keep && at < kEntries; ++at) {
    unsigned long long free = 0;
    if (known[at].compare_exchange_strong(free, key | (unsigned long long)per_sm, std::memory_order_relaxed) ||
        (free & ~0xFFull) == key)
      break;
  }
  return per_sm;
}

}  // namespace gift
