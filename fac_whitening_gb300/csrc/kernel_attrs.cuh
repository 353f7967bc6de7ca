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

}  // namespace gift
