// Layer norm, forward and backward.
//
//   mean = sum(x) / D, rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
//   y = xh w + b with xh = (x - mean) rstd
//   dx = rstd (a - mean(a) - xh mean(a xh)) with a = dy w;  dw = sum dy xh, db = sum dy
//
// Bound by HBM: x and y once forward; x, dy and dx once backward.  A row lives in
// the registers of its threads from its one read to its one write, so the
// variance is the two-pass one (centred squares) without a second read.  Blocks
// are persistent over rows: the parameters are read once per block, and the
// backward's dw and db accumulate in registers over the block's rows, leave one
// partial row per block and are added by column_reduce_kernel in a fixed order.
// What HBM needs in flight (about 60 KB a SM) is more than the row a block works
// on: each thread copies its own vectors of the next rows into a ring in shared
// memory with cp.async, and since it alone reads them back, no barrier is spent on
// the ring.  32768 x 4096 bf16: forward 91 us (5.9 TB/s; 198 us without the ring,
// with 8 elements a thread and every vector checked), backward 142 us (5.7 TB/s); on
// inputs in turn, none of them in L2, 97 and 144, and in fp32 182 and 256 (5.9 and
// 6.3 TB/s).  rsqrtf leaves fp32 rows as near to 64 bits as 1 / sqrtf does (y 6.1e-8).
// What is left is instruction issue (76 and 63 % of the slots are taken).
#include "dense_internal.cuh"

namespace kda {
namespace dense {
namespace {

// How a row is spread: `group` threads (a power of two up to 32, or a multiple
// of 32), each NV vectors of VEC elements, `per_block` rows at once in a block.
struct Split {
  int group, threads, per_block;
};
// The widest row that 512 threads hold: 16 elements each as vectors, 8 one by one
// (16 would not fit the backward's registers).
constexpr int widest(int vec) { return vec > 1 ? 8192 : 4096; }
constexpr int kGroupedWidth = 256;  // up to here a warp or less takes a row

// Sums of the N values over the row's threads; every thread gets them.  Groups
// above a warp go through shared memory: one barrier (two buffers in turn), then
// each thread adds the warps' sums itself.  Shuffles are what these kernels would
// otherwise spend most of their time on: with 8 elements a thread and a second
// tree of shuffles the 4096-wide bf16 forward took 156 us, twice its bytes' time.
template <int N>
struct Sums {
  float v[N];
};
constexpr int kMaxWarps = 32;
template <bool WARPS, int N>
__device__ __forceinline__ Sums<N> row_sum(Sums<N> s, int group, float (*buf)[N][kMaxWarps], int &phase) {
  if constexpr (WARPS) {  // whole warps
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) s.v[n] += __shfl_xor_sync(0xffffffffu, s.v[n], o);
  } else {
    for (int o = min(group, 32) >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) s.v[n] += __shfl_xor_sync(0xffffffffu, s.v[n], o);
    if (group <= 32) return s;
  }
  float(*b)[kMaxWarps] = buf[phase];
  phase ^= 1;
  const int warps = group >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) b[n][threadIdx.x >> 5] = s.v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float a = 0.f;
    for (int w = 0; w < warps; w += 4) {  // the slots past `warps` are zero
      const float4 q = *reinterpret_cast<const float4 *>(&b[n][w]);
      a += (q.x + q.y) + (q.z + q.w);
    }
    s.v[n] = a;
  }
  return s;
}
// Before the first sum: zeros in the slots that no warp writes.
template <int N>
__device__ __forceinline__ void clear_sums(float (*buf)[N][kMaxWarps]) {
  for (int i = threadIdx.x; i < 2 * N * kMaxWarps; i += blockDim.x) (&buf[0][0][0])[i] = 0.f;
  __syncthreads();
}

// Rows of the ring, the current one included: what keeps 60 to 120 KB a SM in
// flight.  Vectors of less than 4 bytes cannot be copied by cp.async: no ring.
template <typename T, int VEC>
constexpr int ring_rows(int nv) {
  return sizeof(T) * VEC < 4 ? 1 : sizeof(T) * VEC * nv <= 64 ? 4 : 3;
}

// A thread's ring of `ROWS` rows of NV vectors; slots of a warp are contiguous.
template <typename T, int VEC, int NV, int ROWS>
struct Ring {
  Vec<T, VEC> *slot;  // this thread's vector 0 of ring row 0
  __device__ __forceinline__ void copy(int k, int i, const T *src) const {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot + (k * NV + i) * (int)blockDim.x);
    if constexpr (sizeof(T) * VEC == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(src) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(to), "l"(src) : "memory");
  }
  __device__ __forceinline__ Vec<T, VEC> get(int k, int i) const {
    return ldvec<T, VEC>(slot[(k * NV + i) * (int)blockDim.x].e);
  }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// WHOLE: a row a block and NV vectors in every thread, so that nothing is checked
// per vector (a third of the instructions otherwise).
template <typename T, int VEC, int NV, bool WHOLE>
__global__ void __launch_bounds__(kMaxThreadsPerRow)
norm_fwd_kernel(Norm P, Split S, T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
  wait_for_stream();
  __shared__ __align__(16) float buf[2][1][kMaxWarps];
  int phase = 0;
  clear_sums<1>(buf);
  const int group = WHOLE ? (int)blockDim.x : S.group;
  const int t = WHOLE ? (int)threadIdx.x : (int)threadIdx.x % group, sub = WHOLE ? 0 : (int)threadIdx.x / group;
  const int D = P.width, nvec = D / VEC;
  const auto has = [&](int i) { return WHOLE || t + i * group < nvec; };
  float w[NV * VEC], b[NV * VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = (t + i * group) * VEC + e;
      w[i * VEC + e] = has(i) && P.weight != nullptr ? ldparam<T>(P.weight, P.param_f32, c) : 1.f;
      b[i * VEC + e] = has(i) && P.bias != nullptr ? ldparam<T>(P.bias, P.param_f32, c) : 0.f;
    }
  const float inv = 1.f / (float)D;
  const int64_t step = (int64_t)gridDim.x * S.per_block;
  constexpr int ROWS = ring_rows<T, VEC>(NV);
  extern __shared__ __align__(16) unsigned char ring_sm[];
  const Ring<T, VEC, NV, ROWS> ring{reinterpret_cast<Vec<T, VEC> *>(ring_sm) + threadIdx.x};
  const T *const x = static_cast<const T *>(P.x) + t * VEC;  // this thread's first vector of row 0
  y += t * VEC;
  const auto fetch = [&](int64_t r, int k) {
    if (r < P.rows) {
      const T *src = x + r * D;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (has(i)) ring.copy(k, i, src + i * group * VEC);
    }
    ring_commit();
  };
  const int64_t r_first = (int64_t)blockIdx.x * S.per_block;
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int k = 0; k < ROWS - 1; ++k) fetch(r_first + k * step + sub, k);
  }
  int k = 0;
#pragma unroll 1
  for (int64_t r0 = r_first; r0 < P.rows; r0 += step) {
    const int64_t r = r0 + sub;
    const bool on = WHOLE || r < P.rows;
    if constexpr (ROWS > 1) {
      fetch(r + (ROWS - 1) * step, k == 0 ? ROWS - 1 : k - 1);
      ring_wait<ROWS - 1>();
    }
    float v[NV * VEC];
    Sums<1> s = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && has(i)) {
        unpack(ROWS > 1 ? ring.get(k, i) : ldvec<T, VEC>(x + r * D + i * group * VEC), v + i * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s.v[0] += v[i * VEC + e];
      }
    }
    k = k + 1 == ROWS ? 0 : k + 1;
    const float mu = row_sum<WHOLE>(s, group, buf, phase).v[0] * inv;
    s.v[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && has(i)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          v[i * VEC + e] -= mu;
          s.v[0] = fmaf(v[i * VEC + e], v[i * VEC + e], s.v[0]);
        }
      }
    }
    const float rs = rsqrtf(row_sum<WHOLE>(s, group, buf, phase).v[0] * inv + P.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && has(i)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          v[i * VEC + e] = fmaf(v[i * VEC + e] * rs, w[i * VEC + e], b[i * VEC + e]);
        stvec<T, VEC>(y + r * D + i * group * VEC, pack<T, VEC>(v + i * VEC));
      }
    }
    if (on && t == 0 && mean != nullptr) {
      mean[r] = mu;
      rstd[r] = rs;
    }
  }
}

// part: [gridDim.x][2][D] partial sums (dw, then db), or NULL when neither is
// wanted; a single block writes the gradients themselves.
template <typename T, int VEC, int NV, bool WHOLE>
__global__ void __launch_bounds__(kMaxThreadsPerRow)
norm_bwd_kernel(Norm P, Split S, const T *__restrict__ dy, const float *__restrict__ mean,
                const float *__restrict__ rstd, T *__restrict__ dx, float *__restrict__ part, void *dweight,
                void *dbias) {
  wait_for_stream();
  // the rings of x and dy; at the end [per_block][2][D] sums when a block works on several rows
  extern __shared__ __align__(16) unsigned char ring_sm[];
  __shared__ __align__(16) float buf[2][2][kMaxWarps];
  int phase = 0;
  clear_sums<2>(buf);
  const int group = WHOLE ? (int)blockDim.x : S.group;
  const int t = WHOLE ? (int)threadIdx.x : (int)threadIdx.x % group, sub = WHOLE ? 0 : (int)threadIdx.x / group;
  const int D = P.width, nvec = D / VEC;
  const auto has = [&](int i) { return WHOLE || t + i * group < nvec; };
  float w[NV * VEC], dw[NV * VEC], db[NV * VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = (t + i * group) * VEC + e;
      w[i * VEC + e] = has(i) && P.weight != nullptr ? ldparam<T>(P.weight, P.param_f32, c) : 1.f;
      dw[i * VEC + e] = db[i * VEC + e] = 0.f;
    }
  const float inv = 1.f / (float)D;
  const int64_t step = (int64_t)gridDim.x * S.per_block;
  constexpr int ROWS = ring_rows<T, VEC>(2 * NV);
  const Ring<T, VEC, 2 * NV, ROWS> ring{reinterpret_cast<Vec<T, VEC> *>(ring_sm) + threadIdx.x};
  const T *const x = static_cast<const T *>(P.x) + t * VEC;  // this thread's first vector of row 0
  dy += t * VEC;
  const auto fetch = [&](int64_t r, int k) {
    if (r < P.rows) {
      const int64_t at = r * D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (has(i)) {
          ring.copy(k, 2 * i, x + at + i * group * VEC);
          ring.copy(k, 2 * i + 1, dy + at + i * group * VEC);
        }
      }
    }
    ring_commit();
  };
  const int64_t r_first = (int64_t)blockIdx.x * S.per_block;
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int k = 0; k < ROWS - 1; ++k) fetch(r_first + k * step + sub, k);
  }
  int slot = 0;
  float mu_next = 0.f, rs_next = 0.f;
  if (r_first + sub < P.rows) mu_next = mean[r_first + sub], rs_next = rstd[r_first + sub];
#pragma unroll 1
  for (int64_t r0 = r_first; r0 < P.rows; r0 += step) {
    const int64_t r = r0 + sub;
    const bool on = WHOLE || r < P.rows;
    if constexpr (ROWS > 1) fetch(r + (ROWS - 1) * step, slot == 0 ? ROWS - 1 : slot - 1);
    const float mu = mu_next, rs = rs_next;
    if (r + step < P.rows) mu_next = mean[r + step], rs_next = rstd[r + step];
    if constexpr (ROWS > 1) ring_wait<ROWS - 1>();
    float xh[NV * VEC], g[NV * VEC];
    Sums<2> s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && has(i)) {
        const int64_t at = r * D + i * group * VEC;
        unpack(ROWS > 1 ? ring.get(slot, 2 * i) : ldvec<T, VEC>(x + at), xh + i * VEC);
        unpack(ROWS > 1 ? ring.get(slot, 2 * i + 1) : ldvec<T, VEC>(dy + at), g + i * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int k = i * VEC + e;
          xh[k] = (xh[k] - mu) * rs;
          dw[k] = fmaf(g[k], xh[k], dw[k]);
          db[k] += g[k];
          g[k] *= w[k];
          s.v[0] += g[k];
          s.v[1] = fmaf(g[k], xh[k], s.v[1]);
        }
      }
    }
    slot = slot + 1 == ROWS ? 0 : slot + 1;
    if (dx == nullptr) continue;
    s = row_sum<WHOLE>(s, group, buf, phase);
    const float m1 = s.v[0] * inv, m2 = s.v[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (on && has(i)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int k = i * VEC + e;
          g[k] = rs * (g[k] - m1 - xh[k] * m2);
        }
        stvec<T, VEC>(dx + t * VEC + r * D + i * group * VEC, pack<T, VEC>(g + i * VEC));
      }
    }
  }
  if (part == nullptr) return;
  float *mine = part + (int64_t)blockIdx.x * 2 * D;
  float *acc_sm = reinterpret_cast<float *>(ring_sm);
  const auto leave = [&](int c, float a, float b) {
    if (gridDim.x > 1) {
      mine[c] = a;
      mine[D + c] = b;
    } else {
      if (dweight != nullptr) stparam<T>(dweight, P.param_f32, c, a);
      if (dbias != nullptr) stparam<T>(dbias, P.param_f32, c, b);
    }
  };
  if (S.per_block == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (has(i))
#pragma unroll
        for (int e = 0; e < VEC; ++e) leave((t + i * group) * VEC + e, dw[i * VEC + e], db[i * VEC + e]);
    return;
  }
  ring_wait<0>();  // the ring's last copies land before its memory takes the sums
  __syncthreads();
  float *to = acc_sm + sub * 2 * D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * group;
    if (has(i))
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        to[c * VEC + e] = dw[i * VEC + e];
        to[D + c * VEC + e] = db[i * VEC + e];
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    float a = 0.f, b = 0.f;
    for (int k = 0; k < S.per_block; ++k) {
      a += acc_sm[k * 2 * D + c];
      b += acc_sm[k * 2 * D + D + c];
    }
    leave(c, a, b);
  }
}

// ---- rows that do not lie on 16-byte boundaries ----
// Element by element the copies alone would take most of the instructions, and
// 2-byte ones cannot be asynchronous.  So the row's enclosing 16-byte pieces are
// copied to the same alignment in shared memory, whole pieces as such, the first
// and the last by the words of the tensor in them, and the threads pick their
// elements there.  The ring is the block's: a barrier a row before it is read.
// Threads and strides are constants, so that addresses are immediates.
constexpr int kOddElems = 8, kOddRows = 4;

template <typename T>
struct RowRing {
  const T *base;        // row 0
  const char *lo, *hi;  // the tensor's bytes
  unsigned char *sm;    // kOddRows slots
  int slot_bytes, D;
  __device__ __forceinline__ static int mis(const T *row) { return (int)((uintptr_t)row & 15); }
  template <int G>
  __device__ __forceinline__ void fetch(int64_t r, int k) const {
    const char *a0 = reinterpret_cast<const char *>(base + r * D), *a1 = a0 + (int64_t)D * sizeof(T);
    const char *from = a0 - mis(base + r * D);
    unsigned char *to = sm + k * slot_bytes;
    const int pieces = (int)(a1 - from + 15) >> 4;
    for (int j = threadIdx.x; j < pieces; j += G) {
      const char *src = from + 16 * j;
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to + 16 * j);
      if (src >= a0 && src + 16 <= a1) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const char *q = src + 4 * w;
          if (q + 4 <= a0 || q >= a1) continue;
          if (q >= lo && q + 4 <= hi) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst + 4 * w), "l"(q) : "memory");
          } else {  // a word with one element of the tensor, at its very start or end
            const char *e = q >= lo ? q : q + sizeof(T);
            *reinterpret_cast<T *>(to + 16 * j + (e - src)) = *reinterpret_cast<const T *>(e);
          }
        }
      }
    }
  }
  __device__ __forceinline__ const T *row(int64_t r, int k) const {
    return reinterpret_cast<const T *>(sm + k * slot_bytes + mis(base + r * D));
  }
};
inline size_t odd_slot(int width, size_t es) { return ((size_t)width * es + 15) / 16 * 16 + 16; }

template <typename T, int G>
__global__ void __launch_bounds__(G)
norm_fwd_odd_kernel(Norm P, T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd, int slot_bytes) {
  wait_for_stream();
  extern __shared__ __align__(16) unsigned char ring_sm[];
  __shared__ __align__(16) float buf[2][1][kMaxWarps];
  int phase = 0;
  clear_sums<1>(buf);
  const int t = threadIdx.x, D = P.width;
  const T *x = static_cast<const T *>(P.x);
  const RowRing<T> ring{x, reinterpret_cast<const char *>(x), reinterpret_cast<const char *>(x + P.rows * D), ring_sm,
                        slot_bytes, D};
  float w[kOddElems], b[kOddElems];
#pragma unroll
  for (int i = 0; i < kOddElems; ++i) {
    const int c = t + i * G;
    w[i] = c < D && P.weight != nullptr ? ldparam<T>(P.weight, P.param_f32, c) : 1.f;
    b[i] = c < D && P.bias != nullptr ? ldparam<T>(P.bias, P.param_f32, c) : 0.f;
  }
  const float inv = 1.f / (float)D;
#pragma unroll
  for (int k = 0; k < kOddRows - 1; ++k) {
    const int64_t r = blockIdx.x + (int64_t)k * gridDim.x;
    if (r < P.rows) ring.template fetch<G>(r, k);
    ring_commit();
  }
  int k = 0;
#pragma unroll 1
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    ring_wait<kOddRows - 2>();
    __syncthreads();  // this row is there for all, and the row before has been read
    const int64_t ahead = r + (int64_t)(kOddRows - 1) * gridDim.x;
    if (ahead < P.rows) ring.template fetch<G>(ahead, k == 0 ? kOddRows - 1 : k - 1);
    ring_commit();
    const T *row = ring.row(r, k) + t;
    k = k + 1 == kOddRows ? 0 : k + 1;
    float v[kOddElems];
    Sums<1> s = {0.f};
#pragma unroll
    for (int i = 0; i < kOddElems; ++i) {
      v[i] = t + i * G < D ? to_f(row[i * G]) : 0.f;
      s.v[0] += v[i];
    }
    const float mu = row_sum<true>(s, G, buf, phase).v[0] * inv;
    s.v[0] = 0.f;
#pragma unroll
    for (int i = 0; i < kOddElems; ++i) {
      v[i] -= mu;
      if (t + i * G < D) s.v[0] = fmaf(v[i], v[i], s.v[0]);
    }
    const float rs = rsqrtf(row_sum<true>(s, G, buf, phase).v[0] * inv + P.eps);
    T *out = y + r * D + t;
#pragma unroll
    for (int i = 0; i < kOddElems; ++i)
      if (t + i * G < D) out[i * G] = from_f<T>(fmaf(v[i] * rs, w[i], b[i]));
    if (t == 0 && mean != nullptr) {
      mean[r] = mu;
      rstd[r] = rs;
    }
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(G)
norm_bwd_odd_kernel(Norm P, const T *__restrict__ dy, const float *__restrict__ mean, const float *__restrict__ rstd,
                    T *__restrict__ dx, float *__restrict__ part, int slot_bytes) {
  wait_for_stream();
  extern __shared__ __align__(16) unsigned char ring_sm[];
  __shared__ __align__(16) float buf[2][2][kMaxWarps];
  int phase = 0;
  clear_sums<2>(buf);
  const int t = threadIdx.x, D = P.width;
  const T *x = static_cast<const T *>(P.x);
  const int64_t all = P.rows * D;
  const RowRing<T> rx{x, reinterpret_cast<const char *>(x), reinterpret_cast<const char *>(x + all), ring_sm,
                      slot_bytes, D};
  const RowRing<T> rd{dy, reinterpret_cast<const char *>(dy), reinterpret_cast<const char *>(dy + all),
                      ring_sm + kOddRows * slot_bytes, slot_bytes, D};
  float w[kOddElems], dw[kOddElems], db[kOddElems];
#pragma unroll
  for (int i = 0; i < kOddElems; ++i) {
    const int c = t + i * G;
    w[i] = c < D && P.weight != nullptr ? ldparam<T>(P.weight, P.param_f32, c) : 1.f;
    dw[i] = db[i] = 0.f;
  }
  const float inv = 1.f / (float)D;
#pragma unroll
  for (int k = 0; k < kOddRows - 1; ++k) {
    const int64_t r = blockIdx.x + (int64_t)k * gridDim.x;
    if (r < P.rows) {
      rx.template fetch<G>(r, k);
      rd.template fetch<G>(r, k);
    }
    ring_commit();
  }
  int k = 0;
  float mu_next = 0.f, rs_next = 0.f;
  if (blockIdx.x < P.rows) mu_next = mean[blockIdx.x], rs_next = rstd[blockIdx.x];
#pragma unroll 1
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const float mu = mu_next, rs = rs_next;
    if (r + gridDim.x < P.rows) mu_next = mean[r + gridDim.x], rs_next = rstd[r + gridDim.x];
    ring_wait<kOddRows - 2>();
    __syncthreads();  // this row is there for all, and the row before has been read
    const int64_t ahead = r + (int64_t)(kOddRows - 1) * gridDim.x;
    if (ahead < P.rows) {
      const int slot = k == 0 ? kOddRows - 1 : k - 1;
      rx.template fetch<G>(ahead, slot);
      rd.template fetch<G>(ahead, slot);
    }
    ring_commit();
    const T *xr = rx.row(r, k) + t, *dr = rd.row(r, k) + t;
    k = k + 1 == kOddRows ? 0 : k + 1;
    float xh[kOddElems], g[kOddElems];
    Sums<2> s = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kOddElems; ++i) {
      const bool on = t + i * G < D;
      g[i] = on ? to_f(dr[i * G]) : 0.f;
      xh[i] = on ? (to_f(xr[i * G]) - mu) * rs : 0.f;
      dw[i] = fmaf(g[i], xh[i], dw[i]);
      db[i] += g[i];
      g[i] *= w[i];
      s.v[0] += g[i];
      s.v[1] = fmaf(g[i], xh[i], s.v[1]);
    }
    if (dx == nullptr) continue;
    s = row_sum<true>(s, G, buf, phase);
    const float m1 = s.v[0] * inv, m2 = s.v[1] * inv;
    T *out = dx + r * D + t;
#pragma unroll
    for (int i = 0; i < kOddElems; ++i)
      if (t + i * G < D) out[i * G] = from_f<T>(rs * (g[i] - m1 - xh[i] * m2));
  }
  if (part == nullptr) return;
  float *mine = part + (int64_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int i = 0; i < kOddElems; ++i)
    if (t + i * G < D) {
      mine[t + i * G] = dw[i];
      mine[D + t + i * G] = db[i];
    }
}

// ---- rows too wide for registers: the row is read again for each pass (from L2) ----
constexpr int kWideThreads = 512;
// VEC parameters from c on: as vectors where they lie on the grid.
template <typename T, int VEC>
__device__ __forceinline__ void param_vec(const Norm &P, const void *p, int c, float none, float *f) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = none;
    return;
  }
  if constexpr (VEC > 1) {
    if (((uintptr_t)p & 15) == 0) {
      if (P.param_f32) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4)
          *reinterpret_cast<float4 *>(f + e) = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c + e));
      } else {
        unpack(ldvec<T, VEC>(static_cast<const T *>(p) + c), f);
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = ldparam<T>(p, P.param_f32, c + e);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads)
norm_fwd_wide_kernel(Norm P, T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
  wait_for_stream();
  __shared__ __align__(16) float buf[2][1][kMaxWarps];
  int phase = 0;
  clear_sums<1>(buf);
  const float inv = 1.f / (float)P.width;
  const int step = blockDim.x * VEC;
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const T *x = static_cast<const T *>(P.x) + r * P.width;
    alignas(16) float f[VEC];
    Sums<1> s = {0.f};
#pragma unroll 2
    for (int c = threadIdx.x * VEC; c < P.width; c += step) {
      unpack(ldvec<T, VEC>(x + c), f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s.v[0] += f[e];
    }
    const float mu = row_sum<true>(s, (int)blockDim.x, buf, phase).v[0] * inv;
    s.v[0] = 0.f;
#pragma unroll 2
    for (int c = threadIdx.x * VEC; c < P.width; c += step) {
      unpack(ldvec<T, VEC>(x + c), f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s.v[0] = fmaf(f[e] - mu, f[e] - mu, s.v[0]);
    }
    const float rs = rsqrtf(row_sum<true>(s, (int)blockDim.x, buf, phase).v[0] * inv + P.eps);
    for (int c = threadIdx.x * VEC; c < P.width; c += step) {
      alignas(16) float w[VEC], b[VEC];
      param_vec<T, VEC>(P, P.weight, c, 1.f, w);
      param_vec<T, VEC>(P, P.bias, c, 0.f, b);
      unpack(ldvec<T, VEC>(x + c), f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = fmaf((f[e] - mu) * rs, w[e], b[e]);
      stvec<T, VEC>(y + r * P.width + c, pack<T, VEC>(f));
    }
    if (threadIdx.x == 0 && mean != nullptr) {
      mean[r] = mu;
      rstd[r] = rs;
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kWideThreads)
norm_bwd_wide_kernel(Norm P, const T *__restrict__ dy, const float *__restrict__ mean,
                     const float *__restrict__ rstd, T *__restrict__ dx) {
  wait_for_stream();
  __shared__ __align__(16) float buf[2][2][kMaxWarps];
  int phase = 0;
  clear_sums<2>(buf);
  const float inv = 1.f / (float)P.width;
  const int step = blockDim.x * VEC;
  for (int64_t r = blockIdx.x; r < P.rows; r += gridDim.x) {
    const T *x = static_cast<const T *>(P.x) + r * P.width, *d = dy + r * P.width;
    const float mu = mean[r], rs = rstd[r];
    alignas(16) float f[VEC], g[VEC], w[VEC];
    Sums<2> s = {0.f, 0.f};
    for (int c = threadIdx.x * VEC; c < P.width; c += step) {
      unpack(ldvec<T, VEC>(x + c), f);
      unpack(ldvec<T, VEC>(d + c), g);
      param_vec<T, VEC>(P, P.weight, c, 1.f, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        g[e] *= w[e];
        s.v[0] += g[e];
        s.v[1] = fmaf(g[e], (f[e] - mu) * rs, s.v[1]);
      }
    }
    s = row_sum<true>(s, (int)blockDim.x, buf, phase);
    const float m1 = s.v[0] * inv, m2 = s.v[1] * inv;
    for (int c = threadIdx.x * VEC; c < P.width; c += step) {
      unpack(ldvec<T, VEC>(x + c), f);
      unpack(ldvec<T, VEC>(d + c), g);
      param_vec<T, VEC>(P, P.weight, c, 1.f, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] = rs * (g[e] * w[e] - m1 - (f[e] - mu) * rs * m2);
      stvec<T, VEC>(dx + r * P.width + c, pack<T, VEC>(g));
    }
  }
}

// dw, db partials of a wide row: thread = a vector of columns, blockIdx.y = slab of rows.
template <typename T, int VEC>
__global__ void __launch_bounds__(128)
norm_param_wide_kernel(Norm P, const T *__restrict__ dy, const float *__restrict__ mean,
                       const float *__restrict__ rstd, float *__restrict__ part) {
  wait_for_stream();
  const int c = (blockIdx.x * 128 + threadIdx.x) * VEC;
  if (c >= P.width) return;
  float dw[VEC], db[VEC], f[VEC], g[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = db[e] = 0.f;
#pragma unroll 4
  for (int64_t r = blockIdx.y; r < P.rows; r += gridDim.y) {
    unpack(ldvec<T, VEC>(static_cast<const T *>(P.x) + r * P.width + c), f);
    unpack(ldvec<T, VEC>(dy + r * P.width + c), g);
    const float mu = mean[r], rs = rstd[r];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      dw[e] = fmaf(g[e], (f[e] - mu) * rs, dw[e]);
      db[e] += g[e];
    }
  }
  float *to = part + (int64_t)blockIdx.y * 2 * P.width + c;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    to[e] = dw[e];
    to[P.width + e] = db[e];
  }
}

constexpr int kWideSlabs = 64;

// Threads of a row off the 16-byte grid: a power of two that holds it at 8 elements each.
int odd_threads(int width) { return width <= 1024 ? 128 : width <= 2048 ? 256 : 512; }

// Rows on the grid, and any of up to 256 elements: 16 elements a thread (fewer
// threads to a row: fewer shuffles), 8 where a warp then holds the row; rows of up
// to 256 elements share a block of 128 threads (4 and more rows at once).
Split split_of(int width, int vec, int *nv) {
  const int units = width / vec;
  const int n = (width > kGroupedWidth ? 16 : 8) / vec;  // vectors a thread
  *nv = n;
  const int need = (units + n - 1) / n;
  Split S;
  if (need <= 32) {
    S.group = 1;
    while (S.group < need) S.group *= 2;
    S.threads = 128;
    S.per_block = S.threads / S.group;
  } else {
    S.group = S.threads = (need + 31) / 32 * 32;
    S.per_block = 1;
  }
  return S;
}

// Persistent blocks: as many as keep `threads` threads a SM in flight and the
// rings within its shared memory.
int blocks_per_sm(const Split &S, int threads, size_t smem) {
  const int by_threads = threads / S.threads;
  const int by_smem = smem > 0 ? (int)((size_t)(220 << 10) / (smem + 1024)) : by_threads;
  const int n = by_threads < by_smem ? by_threads : by_smem;
  return n < 1 ? 1 : n;
}
int64_t grid_of(const Split &S, int64_t rows, int sms, int per_sm) {
  const int64_t blocks = (rows + S.per_block - 1) / S.per_block, most = (int64_t)sms * per_sm;
  return blocks < most ? blocks : most;
}
constexpr int kFwdThreads = 1024, kBwdThreads = 512, kOddBwdThreads = 1024;

template <typename T, int VEC, int NV>
cudaError_t run_fwd(const Norm &P, const Split &S, T *y, float *mean, float *rstd, int sms, cudaStream_t s) {
  constexpr int ROWS = ring_rows<T, VEC>(NV);
  const size_t smem = ROWS > 1 ? sizeof(T) * VEC * NV * ROWS * (size_t)S.threads : 0;
  const bool whole = VEC > 1 && S.per_block == 1 && P.width == S.threads * NV * VEC;
  auto kernel = whole ? norm_fwd_kernel<T, VEC, NV, VEC != 1> : norm_fwd_kernel<T, VEC, NV, false>;
  static std::atomic<int> granted[2][64];  // [whole][device]
  const cudaError_t e = allow_smem(kernel, granted[whole], smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)grid_of(S, P.rows, sms, blocks_per_sm(S, kFwdThreads, smem));
  KDA_LAUNCH("norm_fwd_kernel", s, start_kernel(kernel, grid, S.threads, smem, s, P, S, y, mean, rstd));
  return cudaGetLastError();
}

template <typename T, int VEC, int NV>
cudaError_t run_bwd(const Norm &P, const Split &S, const T *dy, const float *mean, const float *rstd, T *dx,
                    float *part, void *dw, void *db, int *parts, int sms, cudaStream_t s) {
  constexpr int ROWS = ring_rows<T, VEC>(2 * NV);
  const size_t ring = ROWS > 1 ? sizeof(T) * VEC * 2 * NV * ROWS * (size_t)S.threads : 0;
  const size_t sums = part != nullptr && S.per_block > 1 ? sizeof(float) * 2 * P.width * S.per_block : 0;
  const size_t smem = ring > sums ? ring : sums;
  const bool whole = VEC > 1 && S.per_block == 1 && P.width == S.threads * NV * VEC;
  auto kernel = whole ? norm_bwd_kernel<T, VEC, NV, VEC != 1> : norm_bwd_kernel<T, VEC, NV, false>;
  static std::atomic<int> granted[2][64];  // [whole][device]
  const cudaError_t e = allow_smem(kernel, granted[whole], smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)grid_of(S, P.rows, sms, blocks_per_sm(S, kBwdThreads, smem));
  *parts = (int)grid;
  if (grid == 1) *parts = -1;  // the block writes the parameters' gradients
  KDA_LAUNCH("norm_bwd_kernel", s, start_kernel(kernel, grid, S.threads, smem, s, P, S, dy, mean, rstd, dx, part, dw, db));
  return cudaGetLastError();
}

// The kernels for rows off the grid; blocks a SM by threads and by the rings.
template <typename T, int G>
cudaError_t fwd_odd(const Norm &P, T *y, float *mean, float *rstd, int sms, cudaStream_t s) {
  const int slot = (int)odd_slot(P.width, sizeof(T));
  const size_t smem = (size_t)slot * kOddRows;
  static std::atomic<int> granted[64];
  const cudaError_t e = allow_smem(norm_fwd_odd_kernel<T, G>, granted, smem);
  if (e != cudaSuccess) return e;
  const Split S{G, G, 1};
  const unsigned grid = (unsigned)grid_of(S, P.rows, sms, blocks_per_sm(S, kFwdThreads, smem));
  KDA_LAUNCH("norm_fwd_odd_kernel", s, start_kernel(norm_fwd_odd_kernel<T, G>, grid, G, smem, s, P, y, mean, rstd, slot));
  return cudaGetLastError();
}
template <typename T, int G>
cudaError_t bwd_odd(const Norm &P, const T *dy, const float *mean, const float *rstd, T *dx, float *part, int *parts,
                    int sms, cudaStream_t s) {
  const int slot = (int)odd_slot(P.width, sizeof(T));
  const size_t smem = (size_t)slot * kOddRows * 2;
  static std::atomic<int> granted[64];
  const cudaError_t e = allow_smem(norm_bwd_odd_kernel<T, G>, granted, smem);
  if (e != cudaSuccess) return e;
  const Split S{G, G, 1};
  const unsigned grid = (unsigned)grid_of(S, P.rows, sms, blocks_per_sm(S, kOddBwdThreads, smem));
  *parts = (int)grid;
  KDA_LAUNCH("norm_bwd_odd_kernel", s,
             start_kernel(norm_bwd_odd_kernel<T, G>, grid, G, smem, s, P, dy, mean, rstd, dx, part, slot));
  return cudaGetLastError();
}

int vec_of(const Norm &P, const void *a, const void *b) {
  const int vec = P.bf16 ? 8 : 4;
  const uintptr_t bits = (uintptr_t)P.x | (uintptr_t)a | (uintptr_t)b;
  return P.width % vec == 0 && (bits & 15) == 0 ? vec : 1;
}

template <typename T, int VEC>
cudaError_t fwd_wide(const Norm &P, T *y, float *mean, float *rstd, int sms, cudaStream_t s) {
  const unsigned grid = (unsigned)(P.rows < sms * 4 ? P.rows : sms * 4);
  KDA_LAUNCH("norm_fwd_wide_kernel", s, start_kernel(norm_fwd_wide_kernel<T, VEC>, grid, kWideThreads, 0, s, P, y, mean, rstd));
  return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t bwd_wide(const Norm &P, const T *dy, const float *mean, const float *rstd, T *dx, float *part, int *parts,
                     int sms, cudaStream_t s) {
  const unsigned grid = (unsigned)(P.rows < sms * 4 ? P.rows : sms * 4);
  if (dx != nullptr)
    KDA_LAUNCH("norm_bwd_wide_kernel", s, start_kernel(norm_bwd_wide_kernel<T, VEC>, grid, kWideThreads, 0, s, P, dy, mean, rstd, dx));
  if (part != nullptr) {
    *parts = (int)(P.rows < kWideSlabs ? P.rows : kWideSlabs);
    const dim3 pg((unsigned)((P.width + 128 * VEC - 1) / (128 * VEC)), (unsigned)*parts);
    KDA_LAUNCH("norm_param_wide_kernel", s,
               start_kernel(norm_param_wide_kernel<T, VEC>, pg, 128, 0, s, P, dy, mean, rstd, part));
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const Norm &P, T *y, float *mean, float *rstd, int sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int vec = vec_of(P, y, nullptr);
  if (P.width > widest(vec))
    return vec == V ? fwd_wide<T, V>(P, y, mean, rstd, sms, s) : fwd_wide<T, 1>(P, y, mean, rstd, sms, s);
  if (vec == 1 && P.width > kGroupedWidth) {
    const int g = odd_threads(P.width);
    return g == 128   ? fwd_odd<T, 128>(P, y, mean, rstd, sms, s)
           : g == 256 ? fwd_odd<T, 256>(P, y, mean, rstd, sms, s)
                      : fwd_odd<T, 512>(P, y, mean, rstd, sms, s);
  }
  int nv;
  const Split S = split_of(P.width, vec, &nv);
  if (vec == V && nv * V == 8) return run_fwd<T, V, 8 / V>(P, S, y, mean, rstd, sms, s);
  if (vec == V) return run_fwd<T, V, 16 / V>(P, S, y, mean, rstd, sms, s);
  return run_fwd<T, 1, 8>(P, S, y, mean, rstd, sms, s);
}

template <typename T>
cudaError_t bwd(const Norm &P, const T *dy, const float *mean, const float *rstd, T *dx, float *part, void *dw,
                void *db, int *parts, int sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int vec = vec_of(P, dy, dx);
  if (P.width > widest(vec))
    return vec == V ? bwd_wide<T, V>(P, dy, mean, rstd, dx, part, parts, sms, s)
                    : bwd_wide<T, 1>(P, dy, mean, rstd, dx, part, parts, sms, s);
  if (vec == 1 && P.width > kGroupedWidth) {
    const int g = odd_threads(P.width);
    return g == 128   ? bwd_odd<T, 128>(P, dy, mean, rstd, dx, part, parts, sms, s)
           : g == 256 ? bwd_odd<T, 256>(P, dy, mean, rstd, dx, part, parts, sms, s)
                      : bwd_odd<T, 512>(P, dy, mean, rstd, dx, part, parts, sms, s);
  }
  int nv;
  const Split S = split_of(P.width, vec, &nv);
  if (vec == V && nv * V == 8) return run_bwd<T, V, 8 / V>(P, S, dy, mean, rstd, dx, part, dw, db, parts, sms, s);
  if (vec == V) return run_bwd<T, V, 16 / V>(P, S, dy, mean, rstd, dx, part, dw, db, parts, sms, s);
  return run_bwd<T, 1, 8>(P, S, dy, mean, rstd, dx, part, dw, db, parts, sms, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const Norm &P, void *y, float *mean, float *rstd, cudaStream_t s) {
  if (P.rows == 0) return cudaSuccess;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  return P.bf16 ? fwd(P, static_cast<__nv_bfloat16 *>(y), mean, rstd, sms, s)
                : fwd(P, static_cast<float *>(y), mean, rstd, sms, s);
}

// One partial row (dw and db) per block.  The bound counts the blocks without
// their rings' limit and takes the larger of the two vector widths, so that it
// does not depend on the pointers' alignment.
size_t norm_bwd_workspace(const Norm &P) {
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) sms = 152;
  int64_t most = 0;
  for (const int vec : {1, P.bf16 ? 8 : 4}) {
    if (P.width % vec != 0) continue;
    if (P.width > widest(vec)) {
      most = most > kWideSlabs ? most : kWideSlabs;
    } else {
      int nv, g0 = odd_threads(P.width);
      const bool odd = vec == 1 && P.width > kGroupedWidth;
      const Split S = odd ? Split{g0, g0, 1} : split_of(P.width, vec, &nv);
      const int64_t g = grid_of(S, P.rows, sms, blocks_per_sm(S, odd ? kOddBwdThreads : kBwdThreads, 0));
      most = g > most ? g : most;
    }
  }
  return align256(sizeof(float) * 2 * (size_t)P.width * (size_t)most);
}

cudaError_t launch_norm_bwd(const Norm &P, const void *dy, const float *mean, const float *rstd, void *dx,
                            void *dweight, void *dbias, float *part, cudaStream_t s) {
  float *pp = dweight != nullptr || dbias != nullptr ? part : nullptr;
  int parts = 0, sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  typedef __nv_bfloat16 B;
  if (P.rows > 0)
    e = P.bf16 ? bwd(P, static_cast<const B *>(dy), mean, rstd, static_cast<B *>(dx), pp, dweight, dbias, &parts,
                   sms, s)
               : bwd(P, static_cast<const float *>(dy), mean, rstd, static_cast<float *>(dx), pp, dweight, dbias,
                   &parts, sms, s);
  if (e != cudaSuccess || pp == nullptr || parts < 0) return e;  // a single block wrote them itself
  return launch_column_reduce(part, parts, 2 * (int64_t)P.width, P.width, dweight, dbias, P.width, !P.param_f32, s);
}

}  // namespace dense
}  // namespace kda
