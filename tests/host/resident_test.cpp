// The kept occupancy of a kernel answers for the launch that is asked about, whatever was asked before,
// and from several threads.  The runtime's calls are fakes.  Prints "ok", or what went wrong.
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

#include "kernel_attrs.cuh"

namespace {

void kernel_a(int) {}
void kernel_b(int) {}
std::atomic<int> calls{0};

int fits(int threads, int smem) {   // an SM of 2048 threads and 227 KB
  const int by_smem = smem ? 227 * 1024 / smem : 32, by_threads = 2048 / threads;
  return by_smem < by_threads ? by_smem : by_threads;
}

}  // namespace

extern "C" cudaError_t cudaGetDevice(int *dev) {
  *dev = 0;
  return cudaSuccess;
}
extern "C" cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int threads, size_t smem) {
  ++calls;
  *n = fits(threads, (int)smem);
  return cudaSuccess;
}

int check() {
  // one CTA size with no shared memory, a little and a lot, in both orders
  for (int threads : {256, 512, 32})
    for (int smem : {0, 33792, 65536, 0, 65536, 33792, 8192})
      if (gift::resident_per_sm<kernel_a>(threads, smem) != fits(threads, smem)) {
        std::printf("%d threads, %d bytes: %d CTAs, not %d\n", threads, smem,
                    gift::resident_per_sm<kernel_a>(threads, smem), fits(threads, smem));
        return 1;
      }
  return 0;
}

int main() {
  if (check()) return 1;
  const int before = calls;
  std::atomic<int> bad{0};
  std::vector<std::thread> th;
  for (int i = 0; i < 4; ++i) th.emplace_back([&] { bad += check(); });
  for (auto &t : th) t.join();
  if (bad) return 1;
  if (calls != before) {
    std::printf("looked up again what was known: %d calls more\n", calls - before);
    return 1;
  }
  for (int again = 0; again < 2; ++again)   // more sizes than are kept
    for (int smem = 0; smem < 100 * 1024; smem += 1024)
      if (gift::resident_per_sm<kernel_b>(128, smem) != fits(128, smem)) {
        std::printf("%d bytes: not %d CTAs\n", smem, fits(128, smem));
        return 1;
      }
  std::printf("ok\n");
  return 0;
}
