// C entry points of the dense operators: checks of the arguments, then the launchers.
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "dense_internal.cuh"

namespace kda {
namespace dense {
namespace {

kda_status fail(kda_status st, const char *fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_last_error(msg);
  return st;
}

kda_status done(cudaError_t e, const char *where) {
  return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool known(int dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }

kda_status workspace_ok(const void *ws, size_t have, size_t need) {
  if (need == 0) return KDA_OK;
  if (ws == nullptr) return fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (have < need) return fail(KDA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
  if (((uintptr_t)ws & 255) != 0) return fail(KDA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return KDA_OK;
}

// Element alignment: a pointer that is not is no tensor of that type.
bool misaligned(const void *p, bool bf16) { return ((uintptr_t)p & (bf16 ? 1 : 3)) != 0; }

kda_status check_norm(const kda_norm *p, Norm &N) {
  if (p == nullptr) return fail(KDA_ERR_INVALID_ARG, "layer norm: problem is NULL");
  if (p->rows < 0 || p->width < 1)
    return fail(KDA_ERR_INVALID_ARG, "layer norm: rows=%lld width=%d", (long long)p->rows, p->width);
  if (!known(p->dtype) || !known(p->param_dtype))
    return fail(KDA_ERR_INVALID_ARG, "layer norm: unknown dtype %d or param_dtype %d", (int)p->dtype,
                (int)p->param_dtype);
  if (p->dtype == KDA_F32 && p->param_dtype == KDA_BF16)
    return fail(KDA_ERR_UNSUPPORTED, "layer norm: bf16 parameters with fp32 rows");
  if (!(p->eps >= 0.f) || p->eps > 3.0e38f) return fail(KDA_ERR_INVALID_ARG, "layer norm: eps must be finite and >= 0");
  if (p->rows >= ((int64_t)1 << 44) / p->width || p->width > (1 << 26))
    return fail(KDA_ERR_UNSUPPORTED, "layer norm: problem too large");
  if (p->rows > 0 && p->x == nullptr) return fail(KDA_ERR_INVALID_ARG, "layer norm: x is required");
  const bool b = p->dtype == KDA_BF16, pb = p->param_dtype == KDA_BF16;
  if (misaligned(p->x, b) || misaligned(p->weight, pb) || misaligned(p->bias, pb))
    return fail(KDA_ERR_INVALID_ARG, "layer norm: a pointer is not aligned to its element type");
  N = Norm{p->rows, p->width, b, !pb, p->eps, p->x, p->weight, p->bias};
  return KDA_OK;
}

kda_status check_linear(const kda_linear *p, Linear &L) {
  if (p == nullptr) return fail(KDA_ERR_INVALID_ARG, "linear: problem is NULL");
  if (p->rows < 0 || p->outs < 1 || p->ins < 1)
    return fail(KDA_ERR_INVALID_ARG, "linear: rows=%lld outs=%d ins=%d", (long long)p->rows, p->outs, p->ins);
  if (!known(p->dtype)) return fail(KDA_ERR_INVALID_ARG, "linear: unknown dtype %d", (int)p->dtype);
  if ((int)p->activation < KDA_ACT_NONE || (int)p->activation > KDA_ACT_SIGMOID)
    return fail(KDA_ERR_INVALID_ARG, "linear: unknown activation %d", (int)p->activation);
  // no output of more than 2^44 elements: the kernels count their tiles in 32 bits
  const int64_t wide = p->outs > p->ins ? p->outs : p->ins;
  if (p->outs > (1 << 24) || p->ins > (1 << 24) || p->rows > ((int64_t)1 << 30) ||
      p->rows > ((int64_t)1 << 44) / wide || (int64_t)p->outs * p->ins > ((int64_t)1 << 44))
    return fail(KDA_ERR_UNSUPPORTED, "linear: problem too large");
  if (p->weight == nullptr || (p->rows > 0 && p->x == nullptr))
    return fail(KDA_ERR_INVALID_ARG, "linear: x and weight are required");
  const bool b = p->dtype == KDA_BF16;
  if (misaligned(p->x, b) || misaligned(p->weight, b) || misaligned(p->bias, b) || misaligned(p->residual, b))
    return fail(KDA_ERR_INVALID_ARG, "linear: a pointer is not aligned to its element type");
  L = Linear{p->rows, p->outs, p->ins, b, (int)p->activation, p->x, p->weight, p->bias, p->residual};
  return KDA_OK;
}

// What the clipping writes must not overlap: blocks would scale the shared elements
// in no order. Addresses that ascend within a type, as those of views of one flat
// buffer a type do, are checked as they come; others are sorted. With an infinite
// bound what is its own output is not written and does not count.
struct Span {
  uintptr_t begin, end;
  int tensor;
};
kda_status check_outputs(int count, const void *const *in, void *const *out, const int64_t *sizes, const int *dtypes,
                         float max_norm) {
  const bool norm_alone = std::isinf(max_norm);
  const auto written = [&](int i) { return sizes[i] != 0 && !(norm_alone && out[i] == in[i]); };
  const auto span = [&](int i) {
    const uintptr_t p = (uintptr_t)out[i];
    return Span{p, p + (uintptr_t)sizes[i] * (dtypes[i] == KDA_BF16 ? 2 : 4), i};
  };
  uintptr_t first[2] = {0, 0}, end[2] = {0, 0};  // of each type
  int i = 0;
  for (; i < count; ++i) {
    if (!written(i)) continue;
    const Span s = span(i);
    const int t = dtypes[i] == KDA_BF16;
    if (s.begin < end[t]) break;
    if (end[t] == 0) first[t] = s.begin;
    end[t] = s.end;
  }
  if (i == count && (end[0] <= first[1] || end[1] <= first[0])) return KDA_OK;
  const std::unique_ptr<Span[]> all(new (std::nothrow) Span[count]);
  if (all == nullptr) return fail(KDA_ERR_UNSUPPORTED, "clip: no host memory for %d tensors", count);
  int n = 0;
  for (i = 0; i < count; ++i)
    if (written(i)) all[n++] = span(i);
  std::sort(all.get(), all.get() + n, [](const Span &a, const Span &b) {
    return a.begin != b.begin ? a.begin < b.begin : a.tensor < b.tensor;
  });
  for (i = 1; i < n; ++i)
    if (all[i].begin < all[i - 1].end)
      return fail(KDA_ERR_INVALID_ARG, "clip: outputs %d and %d overlap", all[i - 1].tensor, all[i].tensor);
  return KDA_OK;
}

}  // namespace
}  // namespace dense
}  // namespace kda

using namespace kda;
using namespace kda::dense;

extern "C" {

kda_status kda_layer_norm_fwd(const kda_norm *p, void *y, float *mean, float *rstd, void *stream) {
  Norm N{};
  const kda_status st = check_norm(p, N);
  if (st != KDA_OK) return st;
  if (N.rows > 0 && y == nullptr) return fail(KDA_ERR_INVALID_ARG, "layer norm: y is required");
  if ((mean == nullptr) != (rstd == nullptr))
    return fail(KDA_ERR_INVALID_ARG, "layer norm: mean and rstd are kept together or not at all");
  if (misaligned(y, N.bf16) || misaligned(mean, false) || misaligned(rstd, false))
    return fail(KDA_ERR_INVALID_ARG, "layer norm: a pointer is not aligned to its element type");
  return done(launch_norm_fwd(N, y, mean, rstd, (cudaStream_t)stream), "kda_layer_norm_fwd");
}

size_t kda_layer_norm_bwd_workspace_size(const kda_norm *p) {
  Norm N{};
  return check_norm(p, N) == KDA_OK ? norm_bwd_workspace(N) : 0;
}

kda_status kda_layer_norm_bwd(const kda_norm *p, const void *dy, const float *mean, const float *rstd, void *dx,
                              void *dweight, void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
  Norm N{};
  kda_status st = check_norm(p, N);
  if (st != KDA_OK) return st;
  if (N.rows > 0 && (dy == nullptr || mean == nullptr || rstd == nullptr))
    return fail(KDA_ERR_INVALID_ARG, "layer norm: dy, mean and rstd are required");
  if (dx == nullptr && dweight == nullptr && dbias == nullptr)
    return fail(KDA_ERR_INVALID_ARG, "layer norm: no gradient asked for");
  if (misaligned(dy, N.bf16) || misaligned(dx, N.bf16) || misaligned(mean, false) || misaligned(rstd, false) ||
      misaligned(dweight, !N.param_f32) || misaligned(dbias, !N.param_f32))
    return fail(KDA_ERR_INVALID_ARG, "layer norm: a pointer is not aligned to its element type");
  const bool params = dweight != nullptr || dbias != nullptr;
  if ((st = workspace_ok(workspace, workspace_bytes, params ? norm_bwd_workspace(N) : 0)) != KDA_OK) return st;
  return done(launch_norm_bwd(N, dy, mean, rstd, dx, dweight, dbias, static_cast<float *>(workspace),
                              (cudaStream_t)stream),
              "kda_layer_norm_bwd");
}

size_t kda_linear_fwd_workspace_size(const kda_linear *p) {
  Linear L{};
  return check_linear(p, L) == KDA_OK ? linear_fwd_workspace(L) : SIZE_MAX;
}

size_t kda_linear_bwd_workspace_size(const kda_linear *p) {
  Linear L{};
  return check_linear(p, L) == KDA_OK ? linear_bwd_workspace(L) : SIZE_MAX;
}

kda_status kda_linear_fwd(const kda_linear *p, void *y, void *preact, void *workspace, size_t workspace_bytes,
                          void *stream) {
  Linear L{};
  kda_status st = check_linear(p, L);
  if (st != KDA_OK) return st;
  if (L.rows > 0 && y == nullptr) return fail(KDA_ERR_INVALID_ARG, "linear: y is required");
  if (misaligned(y, L.bf16) || misaligned(preact, L.bf16))
    return fail(KDA_ERR_INVALID_ARG, "linear: a pointer is not aligned to its element type");
  if ((st = workspace_ok(workspace, workspace_bytes, linear_fwd_workspace(L))) != KDA_OK) return st;
  return done(launch_linear_fwd(L, y, preact, static_cast<char *>(workspace), (cudaStream_t)stream),
              "kda_linear_fwd");
}

kda_status kda_debug_linear_waits(const kda_linear *p, void *y, void *workspace, size_t workspace_bytes, int *err,
                                  long long polls, void *stream) {
  Linear L{};
  kda_status st = check_linear(p, L);
  if (st != KDA_OK) return st;
  if (!linear_uses_tensor_cores(L)) return fail(KDA_ERR_UNSUPPORTED, "linear waits: not a tensor-core forward");
  if (y == nullptr || err == nullptr || misaligned(y, true) || misaligned(err, false))
    return fail(KDA_ERR_INVALID_ARG, "linear waits: y and err are required");
  if (polls < 0 || polls > umma::kSpinLimit)
    return fail(KDA_ERR_INVALID_ARG, "linear waits: polls must be 0 .. %ld", umma::kSpinLimit);
  if ((st = workspace_ok(workspace, workspace_bytes, linear_fwd_workspace(L))) != KDA_OK) return st;
  return done(launch_linear_fwd(L, y, nullptr, static_cast<char *>(workspace), (cudaStream_t)stream,
                                Waits{(int)polls, err}),
              "kda_debug_linear_waits");
}

kda_status kda_linear_bwd(const kda_linear *p, const void *dy, const void *preact, void *dx, void *dweight,
                          void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
  Linear L{};
  kda_status st = check_linear(p, L);
  if (st != KDA_OK) return st;
  if (dx == nullptr && dweight == nullptr && dbias == nullptr)
    return fail(KDA_ERR_INVALID_ARG, "linear: no gradient asked for");
  if (L.rows > 0 && dy == nullptr) return fail(KDA_ERR_INVALID_ARG, "linear: dy is required");
  if (L.rows > 0 && L.act != KDA_ACT_NONE && preact == nullptr)
    return fail(KDA_ERR_INVALID_ARG, "linear: an activation's backward reads preact");
  if (misaligned(dy, L.bf16) || misaligned(preact, L.bf16) || misaligned(dx, L.bf16) ||
      misaligned(dweight, L.bf16) || misaligned(dbias, L.bf16))
    return fail(KDA_ERR_INVALID_ARG, "linear: a pointer is not aligned to its element type");
  if ((st = workspace_ok(workspace, workspace_bytes, linear_bwd_workspace(L))) != KDA_OK) return st;
  return done(launch_linear_bwd(L, dy, preact, dx, dweight, dbias, static_cast<char *>(workspace),
                                (cudaStream_t)stream),
              "kda_linear_bwd");
}

kda_status kda_linear_status(int **word) {
  if (word == nullptr) return fail(KDA_ERR_INVALID_ARG, "linear status: word is NULL");
  return done(linear_status_word(word), "kda_linear_status");
}

size_t kda_clip_grad_norm_workspace_size(int count) { return count < 0 ? 0 : clip_workspace(count); }

kda_status kda_clip_grad_norm(int count, const void *const *in, void *const *out, const int64_t *sizes,
                              const int *dtypes, float max_norm, float *norm, void *workspace,
                              size_t workspace_bytes, void *stream) {
  if (count < 0 || (count > 0 && (in == nullptr || sizes == nullptr || dtypes == nullptr)))
    return fail(KDA_ERR_INVALID_ARG, "clip: count=%d and its arrays", count);
  if (norm == nullptr || misaligned(norm, false)) return fail(KDA_ERR_INVALID_ARG, "clip: norm is required");
  if (!(max_norm >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "clip: max_norm must be >= 0");
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || !known(dtypes[i]))
      return fail(KDA_ERR_INVALID_ARG, "clip: tensor %d has size %lld, dtype %d", i, (long long)sizes[i], dtypes[i]);
    if (sizes[i] > ((int64_t)1 << 42) || (total += sizes[i]) > ((int64_t)1 << 42))
      return fail(KDA_ERR_UNSUPPORTED, "clip: more than 2^42 elements");
    if (sizes[i] == 0) continue;
    const bool b = dtypes[i] == KDA_BF16;
    if (in[i] == nullptr || misaligned(in[i], b))
      return fail(KDA_ERR_INVALID_ARG, "clip: tensor %d is NULL or misaligned", i);
    if (out != nullptr && (out[i] == nullptr || misaligned(out[i], b)))
      return fail(KDA_ERR_INVALID_ARG, "clip: output %d is NULL or misaligned", i);
  }
  kda_status st = workspace_ok(workspace, workspace_bytes, clip_workspace(count));
  if (st != KDA_OK || (out != nullptr && (st = check_outputs(count, in, out, sizes, dtypes, max_norm)) != KDA_OK)) return st;
  return done(launch_clip(count, in, out, sizes, dtypes, max_norm, norm, static_cast<double *>(workspace),
                          (cudaStream_t)stream),
              "kda_clip_grad_norm");
}

}  // extern "C"
