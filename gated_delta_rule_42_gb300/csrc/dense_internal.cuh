// Definitions shared by the dense operators' translation units (layer norm,
// linear, gradient clipping): problem structs, vector access, launchers.
#pragma once

#include <math.h>

#include <atomic>
#include <mutex>
#include <utility>

#include "kda_internal.cuh"
#include "umma.cuh"

namespace kda {
namespace dense {

constexpr size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr int kMaxThreadsPerRow = 512;

// N elements of T as one 16-byte access (N = 16 / sizeof(T)) or element by element (N = 1).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T e[N];
};
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ldvec(const T *p) {
  Vec<T, N> v;
  if constexpr (sizeof(T) * N == 16) {
    *reinterpret_cast<uint4 *>(v.e) = *reinterpret_cast<const uint4 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v.e[i] = p[i];
  }
  return v;
}
template <typename T, int N>
__device__ __forceinline__ void stvec(T *p, const Vec<T, N> &v) {
  if constexpr (sizeof(T) * N == 16) {
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v.e);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v.e[i];
  }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
// A vector's elements in fp32 and back: two at a time where they are bf16 pairs.
template <typename T, int N>
__device__ __forceinline__ void unpack(const Vec<T, N> &v, float *f) {
  if constexpr (sizeof(T) == 2 && N == 8) {
    const uint4 q = *reinterpret_cast<const uint4 *>(v.e);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(v.e[i]);
  }
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> pack(const float *f) {
  Vec<T, N> v;
  if constexpr (sizeof(T) == 2 && N == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(v.e) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v.e[i] = from_f<T>(f[i]);
  }
  return v;
}
// Element i of a parameter vector held in fp32 or in T.
template <typename T>
__device__ __forceinline__ float ldparam(const void *p, bool f32, int64_t i) {
  return f32 ? static_cast<const float *>(p)[i] : to_f(static_cast<const T *>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void stparam(void *p, bool f32, int64_t i, float x) {
  if (f32)
    static_cast<float *>(p)[i] = x;
  else
    static_cast<T *>(p)[i] = from_f<T>(x);
}

// Lets a kernel take `smem` bytes of dynamic shared memory: the attribute is set
// once per kernel and device (it costs microseconds), again only for more bytes.
// It only ever grows, checked and set under one lock: a call of a smaller size on
// another thread must not take it back between a larger call's grant and launch.
// Up to 40 KB need none, the kernel's static part included.
template <typename K>
cudaError_t allow_smem(K kernel, std::atomic<int> (&granted)[64], size_t smem) {
  if (smem <= (40 << 10)) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (granted[dev].load(std::memory_order_acquire) >= (int)smem) return cudaSuccess;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (granted[dev].load(std::memory_order_relaxed) >= (int)smem) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) granted[dev].store((int)smem, std::memory_order_release);
  return e;
}

// The dense kernels are launched with programmatic stream serialization: a kernel
// is set up while the one before it in the stream ends, and waits at the top for all
// before it to be done, their writes visible. Every kernel launched this way begins
// with that wait, in every thread and before it touches global memory. It saves
// about 2 us between two kernels: the linear step of 1531 x 1001 x 2047 (seven
// kernels) takes 65 us instead of 79, the fp32 one of 2048 x 1024 x 1024 306 instead
// of 324. Releasing the next kernel earlier (griddepcontrol.launch_dependents at the
// top) gained nothing more: 67 and 298 us, the odd norm step 48 instead of 45.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t start_kernel(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         Args &&...args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---- column sums of fp32 partials (reduce.cu) ----
// out[c] = sum over p of part[p * stride + c], c < cols, p < parts, added in a
// fixed order; out in fp32 or bf16, or NULL (skipped).  Two sets in one launch:
// set 1 starts at part + offset1.
cudaError_t launch_column_reduce(const float *part, int parts, int64_t stride, int cols, void *out0, void *out1,
                                 int64_t offset1, bool out_bf16, cudaStream_t s);

// ---- layer norm (norm.cu) ----
struct Norm {
  int64_t rows;
  int width;
  bool bf16, param_f32;
  float eps;
  const void *x, *weight, *bias;
};
cudaError_t launch_norm_fwd(const Norm &P, void *y, float *mean, float *rstd, cudaStream_t s);
size_t norm_bwd_workspace(const Norm &P);
cudaError_t launch_norm_bwd(const Norm &P, const void *dy, const float *mean, const float *rstd, void *dx,
                            void *dweight, void *dbias, float *part, cudaStream_t s);

// ---- gradient clipping (clip.cu) ----
size_t clip_workspace(int count);
cudaError_t launch_clip(int count, const void *const *in, void *const *out, const int64_t *sizes, const int *dtypes,
                        float max_norm, float *norm, double *part, cudaStream_t s);

// ---- linear (linear.cu, linear_simt.cu) ----
// The activations: value and slope.  The fp32 path calls CUDA's functions, the
// normal distribution as erfc (1 + erf cancels for negative z: 4 % off at z = -5).
// The bf16 path (FAST) takes the hardware exponential and, for erfc, the rational
// approximation 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical
// Functions, at a third of the instructions; its e^(-z^2/2) is the one the slope
// needs as well.  Its error of 1.5e-7 is an absolute one: below half a step of
// bf16 (2^-8 of the value) down to z = -6, where gelu is -6e-9, and 1 % of gelu's
// -5e-15 at z = -8.
// The exponential and the reciprocal flush denormals: what would be one rounds to
// nothing beside the terms it is added to, and the handling costs more than both.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_fast(1.f + exp2_fast(-kLog2e * z)); }
// (Phi(z), e^(-z^2/2)), Phi the normal distribution function
__device__ __forceinline__ float2 normal_fast(float z) {
  const float g = exp2_fast(-0.5f * kLog2e * z * z);
  const float t = rcp_fast(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
  float p = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  p = fmaf(p, t, 0.5f * 1.421413741f);
  p = fmaf(p, t, 0.5f * -0.284496736f);
  p = fmaf(p, t, 0.5f * 0.254829592f);
  const float half_erfc = p * t * g;  // of |z| / sqrt 2
  return make_float2(z < 0.f ? half_erfc : 1.f - half_erfc, g);
}
template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == KDA_ACT_SILU) return FAST ? z * sigmoid_fast(z) : z / (1.f + expf(-z));
  if constexpr (ACT == KDA_ACT_GELU)
    return FAST ? z * normal_fast(z).x : 0.5f * z * erfcf(z * -0.70710678118654752f);
  if constexpr (ACT == KDA_ACT_SIGMOID) return FAST ? sigmoid_fast(z) : 1.f / (1.f + expf(-z));
  return z;
}
template <int ACT, bool FAST>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == KDA_ACT_SILU) {
    const float p = FAST ? sigmoid_fast(z) : 1.f / (1.f + expf(-z));
    return p * (1.f + z * (1.f - p));
  }
  if constexpr (ACT == KDA_ACT_GELU) {
    if (FAST) {
      const float2 n = normal_fast(z);
      return fmaf(z * 0.39894228040143268f, n.y, n.x);
    }
    return 0.5f * erfcf(z * -0.70710678118654752f) + z * 0.39894228040143268f * expf(-0.5f * z * z);
  }
  if constexpr (ACT == KDA_ACT_SIGMOID) {
    // e / (1 + e)^2 with e = e^-|z|: p (1 - p) cancels for large z (17 % off at z = 15 in fp32, 0 from 17 on)
    if (FAST) {
      const float e = exp2_fast(-kLog2e * fabsf(z)), r = rcp_fast(1.f + e);
      return e * r * r;
    }
    const float e = expf(-fabsf(z)), d = 1.f + e;
    return e / (d * d);
  }
  return 1.f;
}

// C(m, n) = sum over k of A(m, k) B(n, k), then the epilogue
// z = C + bias[n], y = act(z) + residual(m, n).  Element (m, k) of an operand is
// p[m * ld + k] (k_major) or p[k * ld + m].  Rows of y, preact and residual are
// N elements apart.
struct Operand {
  const void *p;
  int64_t ld;
  bool k_major;
};
struct Product {
  int64_t M, N, K;
  Operand a, b;
  const void *bias, *residual;  // or NULL
  int act;
  void *y, *preact;  // preact or NULL
};


struct Linear {
  int64_t rows;
  int outs, ins;
  bool bf16;
  int act;
  const void *x, *weight, *bias, *residual;
};
// The bounds of a tensor-core product's waits: polls each, and the device word that
// a wait that gave up sets to 1 (NULL: the library's own, linear_status_word).
struct Waits {
  int polls;
  int *err;
};
constexpr Waits kWaits{(int)umma::kSpinLimit, nullptr};
// Device word that is nonzero once a bounded wait of a product gave up.
cudaError_t linear_status_word(int **p);
size_t linear_fwd_workspace(const Linear &L);
size_t linear_bwd_workspace(const Linear &L);
cudaError_t launch_linear_fwd(const Linear &L, void *y, void *preact, char *ws, cudaStream_t s,
                              const Waits &waits = kWaits);
bool linear_uses_tensor_cores(const Linear &L);  // its forward
cudaError_t launch_linear_bwd(const Linear &L, const void *dy, const void *preact, void *dx, void *dweight,
                              void *dbias, char *ws, cudaStream_t s);

}  // namespace dense
}  // namespace kda
