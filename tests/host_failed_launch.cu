// Sequences of launches, without a GPU: the runtime's launch is replaced by one that
// fails at the n-th call. Nothing may be launched after a failure, and the call returns it.
#include <cuda_runtime.h>

#include <cstdio>
#include <vector>

int launches = 0, fail_at = 0;
cudaError_t last_error = cudaSuccess;
template <typename... Args>
cudaError_t fake_launch(const cudaLaunchConfig_t *, Args &&...) {
  if (++launches == fail_at) last_error = cudaErrorLaunchOutOfResources;
  return last_error;
}
cudaError_t take_error() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}
#define cudaLaunchKernelEx fake_launch
#define cudaGetLastError take_error
#include "clip.cu"
#include "linear_simt.cu"

namespace kda {
void inst_begin(const char *, cudaStream_t) {}
void inst_end(cudaStream_t) {}
cudaError_t sm_count(int *n) { return *n = 152, cudaSuccess; }
}  // namespace kda

template <typename F>
int check(const char *name, int expected, F call) {
  for (fail_at = 0; fail_at <= expected; ++fail_at) {
    launches = 0;
    const cudaError_t e = call();
    const int want = fail_at ? fail_at : expected;
    if (launches != want || (e != cudaSuccess) != (fail_at != 0) || last_error != cudaSuccess) {
      std::printf("%s: failing at %d of %d: %d launches, error %d\n", name, fail_at, expected, launches, (int)e);
      return 1;
    }
  }
  return 0;
}

int main() {
  using namespace kda::dense;
  alignas(16) static float buffer[4];
  const int count = 2500;  // three tables
  std::vector<const void *> in(count, buffer);
  std::vector<void *> out(count, buffer);
  std::vector<int64_t> sizes(count, 4);
  std::vector<int> kinds(count, KDA_F32);
  float norm;
  double part[1];
  int bad = check("clip", 6, [&] {
    return launch_clip(count, in.data(), out.data(), sizes.data(), kinds.data(), 1.f, &norm, part, nullptr);
  });
  bad += check("clip, norm alone", 4, [&] {
    return launch_clip(count, in.data(), nullptr, sizes.data(), kinds.data(), 1.f, &norm, part, nullptr);
  });
  // 128 tiles of 128 x 128 in equal runs over two blocks a SM: a product and a join
  const Product P{2048, 1024, 1024, {buffer, 1024, true}, {buffer, 1024, true}, nullptr, nullptr, KDA_ACT_SILU, buffer,
                  nullptr};
  bad += check("fp32 product", 2, [&] { return launch_simt(P, buffer, 152, nullptr); });
  return bad;
}
