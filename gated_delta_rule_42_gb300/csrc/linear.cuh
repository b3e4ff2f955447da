// Pieces shared by the linear layer's kernels: the epilogue of one output, the
// split of the k axis and the choice of an activation's instance.
#pragma once

#include "dense_internal.cuh"

namespace kda {
namespace dense {

// The epilogue of output (m, n) with the product's sum c.
template <typename T, int ACT>
__device__ __forceinline__ void finish_one(const Product &P, int64_t m, int64_t n, float c) {
  if (P.bias != nullptr) c += to_f(static_cast<const T *>(P.bias)[n]);
  const int64_t at = m * P.N + n;
  if (P.preact != nullptr) static_cast<T *>(P.preact)[at] = from_f<T>(c);
  c = act_value<ACT, sizeof(T) == 2>(c);
  if (P.residual != nullptr) c += to_f(static_cast<const T *>(P.residual)[at]);
  static_cast<T *>(P.y)[at] = from_f<T>(c);
}

// Eight bf16 outputs of one row, as 16-byte accesses (see rows_on_grid): c is
// the sums with the bias added, res the residual's values where there is one.
template <int ACT>
__device__ __forceinline__ void finish_8(const Product &P, int64_t at, float (&c)[8],
                                         const Vec<__nv_bfloat16, 8> &res) {
  typedef __nv_bfloat16 B;
  if (P.preact != nullptr) stvec<B, 8>(static_cast<B *>(P.preact) + at, pack<B, 8>(c));
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = act_value<ACT, true>(c[e]);
  if (P.residual != nullptr) {
    float r[8];
    unpack(res, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] += r[e];
  }
  stvec<B, 8>(static_cast<B *>(P.y) + at, pack<B, 8>(c));
}
// Eight values of the bias from n on (a multiple of 8 below P.N), or zeros.
__device__ __forceinline__ void bias_8(const Product &P, int64_t n, float (&b)[8]) {
  if (P.bias == nullptr || n >= P.N) {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = 0.f;
    return;
  }
  unpack(ldvec<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(P.bias) + n), b);
}

// Whether every output row and what is read beside it lie on 16-byte boundaries.
inline bool rows_on_grid(const Product &P) {
  const uintptr_t bits = (uintptr_t)P.y | (uintptr_t)P.preact | (uintptr_t)P.residual | (uintptr_t)P.bias;
  return P.N % 8 == 0 && (bits & 15) == 0;
}

// Runs the statement with the constexpr int ACT of a checked activation.
#define DENSE_ACT_SWITCH(act, ...)           \
  switch (act) {                             \
    case KDA_ACT_SILU: {                     \
      constexpr int ACT = KDA_ACT_SILU;      \
      __VA_ARGS__;                           \
    } break;                                 \
    case KDA_ACT_GELU: {                     \
      constexpr int ACT = KDA_ACT_GELU;      \
      __VA_ARGS__;                           \
    } break;                                 \
    case KDA_ACT_SIGMOID: {                  \
      constexpr int ACT = KDA_ACT_SIGMOID;   \
      __VA_ARGS__;                           \
    } break;                                 \
    default: {                               \
      constexpr int ACT = KDA_ACT_NONE;      \
      __VA_ARGS__;                           \
    } break;                                 \
  }

// Product of the fp32 pipes (linear_simt.cu), K >= 1, the epilogue included; part:
// simt_part_bytes of workspace.
size_t simt_part_bytes(int64_t M, int64_t N, int64_t K, int sms);
cudaError_t launch_simt(const Product &P, float *part, int sms, cudaStream_t s);

// Product of a few fp32 rows: M <= kFewRows32, both operands with k contiguous and
// rows K apart; no workspace.
constexpr int kFewRows32 = 16;
cudaError_t launch_few32(const Product &P, cudaStream_t s);

// Product of the tensor cores (linear_tc.cu): bf16 operands whose base and rows
// lie on 16-byte boundaries, K >= 1, the epilogue and the join included.
size_t tc_part_bytes(int64_t M, int64_t N, int64_t K, int sms);
cudaError_t launch_tc(const Product &P, float *part, int sms, cudaStream_t s, const Waits &waits);

// Product of a few rows (linear_few.cu): bf16, M <= kFewRows, both operands with
// k contiguous and rows K apart (any alignment); no workspace.
constexpr int kFewRows = 32;
cudaError_t launch_few(const Product &P, cudaStream_t s);

}  // namespace dense
}  // namespace kda
