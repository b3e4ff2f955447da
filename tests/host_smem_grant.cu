// The grant of dynamic shared memory under two host threads, without a GPU: the
// runtime's calls are replaced, and the one for the smaller size is held up until the
// larger size has been set (200 ms at most, since a lock may keep the other out).
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

constexpr int kSmall = 64 << 10, kLarge = 128 << 10;
std::atomic<int> attribute{0};
std::atomic<bool> small_inside{false};

cudaError_t set_attribute(int bytes) {
  if (bytes == kSmall) {
    small_inside = true;
    for (int i = 0; i < 200 && attribute < kLarge; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  }
  attribute = bytes;
  return cudaSuccess;
}
#define cudaFuncSetAttribute(kernel, which, bytes) set_attribute(bytes)
#define cudaGetDevice(p) (*(p) = 0, cudaSuccess)
#include "dense_internal.cuh"

void kernel() {}

int main() {
  std::atomic<int> granted[64] = {};
  std::thread small([&] { kda::dense::allow_smem(kernel, granted, kSmall); });
  while (!small_inside) std::this_thread::yield();
  std::thread large([&] { kda::dense::allow_smem(kernel, granted, kLarge); });
  large.join();
  small.join();
  // both were told that they may launch
  std::printf("attribute %d granted %d\n", attribute.load(), granted[0].load());
  if (attribute < kLarge || granted[0] > attribute) return 1;
  kda::dense::allow_smem(kernel, granted, kSmall);
  return attribute < kLarge ? 2 : 0;
}
