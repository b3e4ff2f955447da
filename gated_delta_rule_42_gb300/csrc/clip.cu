// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over all tensors of g^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// Bound by HBM: every gradient is read for the norm, and read and written for
// the scaling, which can start only when the whole norm is known.  The tensors
// travel as a table in the kernel's parameters (no copy to the device, nothing
// kept between calls), cut into chunks of 8192 elements.  Each block has a
// contiguous run of chunks, so that it searches the table once and then steps
// along it.  The second pass gives the blocks the same runs, from the end: what the
// first pass read last is still in L2.  1.34 G elements (2.7 GB of bf16): 405 us for
// the norm (6.6 TB/s), 840 us for the scaling (6.4 TB/s).  With chunks of 4096, and
// so half the loads in flight, the norm took 525 us (417 with 8192 at the time).
#include "dense_internal.cuh"

namespace kda {
namespace dense {
namespace {

constexpr int kChunkElems = 8192;
constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;
constexpr int kMaxBlocks = 2048;  // partial sums of one launch

// A launch's tensors: 28 bytes each; the parameter space of a launch is 32,764 bytes.
template <int CAP>
struct Table {
  const void *in[CAP];
  void *out[CAP];
  int64_t size[CAP];  // elements, and kBf16
  int first[CAP];     // a tensor's first chunk within the launch
  int count, chunks;
};
constexpr int64_t kBf16 = (int64_t)1 << 62;
constexpr int kSmallTable = 60, kMediumTable = 250, kLargeTable = 1000;

// The tensor that holds a chunk: the last one whose first chunk is not past it
// (the table has no empty tensors).
template <int CAP>
__device__ __forceinline__ int find(const Table<CAP> &tab, int chunk) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}
// A block's run of chunks [begin, end).
template <int CAP>
__device__ __forceinline__ void run_of(const Table<CAP> &tab, int *begin, int *end) {
  *begin = (int)((int64_t)tab.chunks * blockIdx.x / gridDim.x);
  *end = (int)((int64_t)tab.chunks * (blockIdx.x + 1) / gridDim.x);
}
// Chunk c of tensor i: its first element and its length.
template <int CAP>
__device__ __forceinline__ int chunk_of(const Table<CAP> &tab, int i, int c, int64_t *at) {
  *at = (int64_t)(c - tab.first[i]) * kChunkElems;
  const int64_t left = (tab.size[i] & ~kBf16) - *at;
  return (int)(left < kChunkElems ? left : kChunkElems);
}

// A whole aligned chunk is read in batches of four 16-byte loads a thread, issued
// together: with 8 blocks a SM that is 128 KB a SM in flight.
constexpr int kBatch = 4;

// Squares are taken in fp32.  A thread's sum of up to 32 of them is kept where no
// square can have overflowed, and none that counts beside the sum can have lost
// bits below 2^-126; where it lies outside, the same elements are scaled by a power
// of two and squared again, and the scale's square is taken out in fp64.  Elements
// anywhere in fp32's range then count at full accuracy, and ordinary gradients pay
// one comparison a sum (24 matrices of 4096 x 4096 bf16: 158 us, zeros 160).
constexpr float kSumMin = 0x1p-96f, kSumMax = 0x1p120f;
__device__ __forceinline__ bool in_range(float a) { return a >= kSumMin && a <= kSumMax; }
// Below: 2^100, so that 2^-149 has a square of 2^-98; above, or not a number: 2^-80,
// so that the largest value's square is 2^96.
__device__ __forceinline__ float rescale_of(float a) { return a < kSumMin ? 0x1p100f : 0x1p-80f; }
__device__ __forceinline__ double unscaled(float sum, float scale) {
  return (double)sum * (scale > 1.f ? 0x1p-200 : 0x1p160);
}

// The squares of p[0, n) that are this thread's, n < kChunkElems or p off the
// 16-byte grid, each element multiplied by `scale` first (1 changes nothing).
template <typename T>
__device__ __forceinline__ float part_squares(const T *p, int n, float scale) {
  constexpr int V = 16 / sizeof(T);
  float a = 0.f;
  int i0 = 0;
  if (((uintptr_t)p & 15) == 0) {
    const int nv = n / V;
    for (int i = threadIdx.x; i < nv; i += kThreads) {
      float f[V];
      unpack(ldvec<T, V>(p + i * V), f);
#pragma unroll
      for (int e = 0; e < V; ++e) a = fmaf(f[e] * scale, f[e] * scale, a);
    }
    i0 = nv * V;
  }
  for (int i = i0 + threadIdx.x; i < n; i += kThreads) {
    const float f = to_f(p[i]) * scale;
    a = fmaf(f, f, a);
  }
  return a;
}
// The squares of a batch of vectors.
template <typename T>
__device__ __forceinline__ float batch_squares(const Vec<T, 16 / sizeof(T)> (&u)[kBatch], float scale) {
  constexpr int V = 16 / sizeof(T);
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    float f[V];
    unpack(u[k], f);
#pragma unroll
    for (int e = 0; e < V; ++e) a = fmaf(f[e] * scale, f[e] * scale, a);
  }
  return a;
}
template <typename T>
__device__ __forceinline__ bool all_zero(const Vec<T, 16 / sizeof(T)> (&u)[kBatch]) {
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const uint4 q = *reinterpret_cast<const uint4 *>(u[k].e);
    bits |= q.x | q.y | q.z | q.w;
  }
  return (bits & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu)) == 0;  // zeros of either sign
}

// Sum of squares of n elements (n <= kChunkElems) over the block's threads.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int n) {
  constexpr int V = 16 / sizeof(T);
  if (n == kChunkElems && ((uintptr_t)p & 15) == 0) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kChunkElems / V / kThreads; j += kBatch) {
      Vec<T, V> u[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) u[k] = ldvec<T, V>(p + ((j + k) * kThreads + threadIdx.x) * V);
      const float a = batch_squares<T>(u, 1.f);
      if (in_range(a)) {
        sum += (double)a;
      } else if (!all_zero<T>(u)) {  // still in registers
        const float scale = rescale_of(a);
        sum += unscaled(batch_squares<T>(u, scale), scale);
      }
    }
    return sum;
  }
  const float a = part_squares(p, n, 1.f);
  if (in_range(a)) return (double)a;
  const float scale = rescale_of(a);
  return unscaled(part_squares(p, n, scale), scale);
}

template <typename T>
__device__ __forceinline__ Vec<T, 16 / sizeof(T)> scaled(const Vec<T, 16 / sizeof(T)> &u, float s) {
  constexpr int V = 16 / sizeof(T);
  float f[V];
  unpack(u, f);
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] *= s;
  return pack<T, V>(f);
}

// p and q may be the same: a thread writes only what it has read.
template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *q, int n, float s) {
  constexpr int V = 16 / sizeof(T);
  int i0 = 0;
  if ((((uintptr_t)p | (uintptr_t)q) & 15) == 0) {
    if (n == kChunkElems) {
#pragma unroll
      for (int j = 0; j < kChunkElems / V / kThreads; j += kBatch) {
        Vec<T, V> u[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) u[k] = ldvec<T, V>(p + ((j + k) * kThreads + threadIdx.x) * V);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) stvec<T, V>(q + ((j + k) * kThreads + threadIdx.x) * V, scaled<T>(u[k], s));
      }
      return;
    }
    const int nv = n / V;
    for (int i = threadIdx.x; i < nv; i += kThreads) stvec<T, V>(q + i * V, scaled<T>(ldvec<T, V>(p + i * V), s));
    i0 = nv * V;
  }
  for (int i = i0 + threadIdx.x; i < n; i += kThreads) q[i] = from_f<T>(to_f(p[i]) * s);
}

// Block sum in fp64, the same order whatever the timing; every thread gets it.
__device__ __forceinline__ double block_sum(double a) {
  __shared__ double sm[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = a;
  __syncthreads();
  a = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) a += sm[w];
  return a;
}

// part[blockIdx.x] = the sum of squares of the block's chunks: fp32 within a
// thread's batch (32 elements at most), fp64 beyond.
template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const __grid_constant__ Table<CAP> tab, double *part) {
  wait_for_stream();
  double a = 0.0;
  int c, end;
  run_of(tab, &c, &end);
  int i = find(tab, c);
  for (; c < end; ++c) {
    if (i + 1 < tab.count && c >= tab.first[i + 1]) ++i;
    int64_t at;
    const int n = chunk_of(tab, i, c, &at);
    a += tab.size[i] & kBf16 ? chunk_squares(static_cast<const __nv_bfloat16 *>(tab.in[i]) + at, n)
                             : chunk_squares(static_cast<const float *>(tab.in[i]) + at, n);
  }
  a = block_sum(a);
  if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// Every block adds the partial sums itself (the same order in each), then scales its chunks.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
clip_scale_kernel(const __grid_constant__ Table<CAP> tab, const double *__restrict__ part, int parts, float max_norm,
                  float *norm) {
  wait_for_stream();
  double a = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) a += part[i];
  a = sqrt(block_sum(a));
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)a;
  const double ratio = (double)max_norm / (a + 1e-6);
  // an infinite bound scales nothing; otherwise NaN stays NaN
  const float s = ratio >= 1.0 || isinf(max_norm) ? 1.f : (float)ratio;
  if (tab.chunks == 0) return;
  int begin, c;
  run_of(tab, &begin, &c);
  int i = find(tab, --c);
  for (; c >= begin; --c) {
    if (c < tab.first[i]) --i;
    if (s == 1.f && tab.out[i] == tab.in[i]) continue;  // in place and nothing to scale
    int64_t at;
    const int n = chunk_of(tab, i, c, &at);
    if (tab.size[i] & kBf16)
      chunk_scale(static_cast<const __nv_bfloat16 *>(tab.in[i]) + at, static_cast<__nv_bfloat16 *>(tab.out[i]) + at, n, s);
    else
      chunk_scale(static_cast<const float *>(tab.in[i]) + at, static_cast<float *>(tab.out[i]) + at, n, s);
  }
}

int64_t chunks_of(int64_t size) { return (size + kChunkElems - 1) / kChunkElems; }

// Walks the non-empty tensors a table at a time (all chunks together fit an int:
// the entry point refuses more than 2^42 elements).
struct Walk {
  int count;
  const void *const *in;
  void *const *out;
  const int64_t *sizes;
  const int *dtypes;
  int at = 0;
  template <int CAP>
  bool next(Table<CAP> &tab) {
    tab.count = tab.chunks = 0;
    for (; at < count && tab.count < CAP; ++at) {
      if (sizes[at] == 0) continue;
      tab.in[tab.count] = in[at];
      tab.out[tab.count] = out != nullptr ? out[at] : nullptr;
      tab.size[tab.count] = sizes[at] | (dtypes[at] == KDA_BF16 ? kBf16 : 0);
      tab.first[tab.count++] = tab.chunks;
      tab.chunks += (int)chunks_of(sizes[at]);
    }
    return tab.count > 0;
  }
};

template <int CAP>
cudaError_t run(Walk w, int sms, float max_norm, float *norm, double *part, cudaStream_t s) {
  const int most = sms * kBlocksPerSm < kMaxBlocks ? sms * kBlocksPerSm : kMaxBlocks;
  Table<CAP> tab;
  int parts = 0;
  Walk again = w;
  cudaError_t e;  // a pass that was not launched leaves nothing to scale by: the call ends there
  while (w.next(tab)) {
    const int grid = tab.chunks < most ? tab.chunks : most;
    KDA_LAUNCH("clip_norm_kernel", s, start_kernel(clip_norm_kernel<CAP>, grid, kThreads, 0, s, tab, part + parts));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    parts += grid;
  }
  bool first = true;
  while (again.next(tab) || first) {
    if (again.out == nullptr) tab.chunks = 0;  // the norm alone
    const int grid = tab.chunks < 1 ? 1 : tab.chunks < most ? tab.chunks : most;
    KDA_LAUNCH("clip_scale_kernel", s,
               start_kernel(clip_scale_kernel<CAP>, grid, kThreads, 0, s, tab, part, parts, max_norm, first ? norm : nullptr));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    first = false;
    if (again.out == nullptr) break;
  }
  return cudaSuccess;
}

}  // namespace

// kMaxBlocks partial sums a launch, one launch for every kLargeTable tensors.
size_t clip_workspace(int count) { return align256(sizeof(double) * kMaxBlocks * (size_t)(count / kLargeTable + 1)); }

cudaError_t launch_clip(int count, const void *const *in, void *const *out, const int64_t *sizes, const int *dtypes,
                        float max_norm, float *norm, double *part, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const Walk w{count, in, out, sizes, dtypes};
  // the parameters cost their bytes at every launch: the smallest table that holds the tensors
  if (count <= kSmallTable) return run<kSmallTable>(w, sms, max_norm, norm, part, s);
  if (count <= kMediumTable) return run<kMediumTable>(w, sms, max_norm, norm, part, s);
  return run<kLargeTable>(w, sms, max_norm, norm, part, s);
}

}  // namespace dense
}  // namespace kda
