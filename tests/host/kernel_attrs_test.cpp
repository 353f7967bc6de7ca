// The host's per-kernel state under two threads, with the CUDA runtime's calls replaced by fakes.
// Prints "ok", or what went wrong.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include "kernel_attrs.cuh"

namespace {

void kernel_a(int) {}

std::atomic<int> limit{0};         // the kernel's attribute
std::atomic<int> calls{0};         // of the attribute call
std::atomic<bool> first_in{false}, second_set{false}, first_back{false};

// for half a second at most
void until(const std::atomic<bool> &flag) {
  for (int i = 0; i < 500 && !flag; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
}

}  // namespace

extern "C" cudaError_t cudaGetDevice(int *dev) {
  *dev = 0;
  return cudaSuccess;
}

// The order that two threads may meet in: the first caller's value (the smaller) is set after the second's,
// and the second call returns after the first thread has gone on.
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
  if (calls++ == 0) {
    first_in = true;
    until(second_set);
    limit = bytes;
  } else {
    limit = bytes;
    second_set = true;
    until(first_back);
  }
  return cudaSuccess;
}

int main() {
  constexpr int small = 50688, large = 63360;   // one kernel with CTAs of 12 and of 15 warps
  std::thread a([] {
    gift::ensure_dynamic_smem<kernel_a>(small);
    first_back = true;
  });
  while (!first_in) std::this_thread::yield();
  std::thread b([] { gift::ensure_dynamic_smem<kernel_a>(large); });
  a.join();
  b.join();
  if (gift::ensure_dynamic_smem<kernel_a>(large) != cudaSuccess || limit < large) {
    std::printf("the limit is %d bytes for a launch of %d\n", limit.load(), large);
    return 1;
  }
  const int before = calls;
  if (gift::ensure_dynamic_smem<kernel_a>(small) != cudaSuccess || calls != before || limit < large) {
    std::printf("a smaller request called again or lowered the limit to %d bytes\n", limit.load());
    return 1;
  }
  std::printf("ok\n");
  return 0;
}
