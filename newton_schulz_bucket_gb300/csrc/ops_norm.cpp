// The layer norm and the balance loss behind the C ABI (include/muon_ops.h):
// argument checks and launches.
#include <cmath>

#include "ops_checks.h"

using namespace muon;

namespace {

muon_status_t check_norm(const char* what, const NormArgs& a) {
  if (!dtype_ok(a.dtype)) return fail(MUON_ERR_INVALID_ARG, "%s: dtype is not a muon_dtype_t", what);
  if (a.w_dtype != a.dtype && a.w_dtype != DT_F32)
    return fail(MUON_ERR_INVALID_ARG, "%s: w_dtype must be dtype or F32", what);
  if (a.rows < 0 || a.rows > kMaxDim || a.width < 1 || a.width > kMaxDim)
    return fail(MUON_ERR_INVALID_ARG, "%s: rows must be in [0, 2^30], width in [1, 2^30]", what);
  return MUON_OK;
}
muon_status_t check_pitch(const char* what, int64_t stride, int64_t width) {
  if (stride < width || stride > kMaxStride)
    return fail(MUON_ERR_INVALID_ARG, "%s: a row stride must be in [width, 2^36]", what);
  return MUON_OK;
}
// The parts' sums over rows: dw and db of every column, fp32.
size_t norm_bytes(int64_t rows, int64_t width) {
  return align256((size_t)norm_part_rows(rows, width) * 2 * width * sizeof(float));
}

muon_status_t check_balance(const char* what, const BalanceArgs& a) {
  if (!dtype_ok(a.dtype)) return fail(MUON_ERR_INVALID_ARG, "%s: dtype is not a muon_dtype_t", what);
  if (a.tokens < 0 || a.tokens > kMaxDim) return fail(MUON_ERR_INVALID_ARG, "%s: tokens must be in [0, 2^30]", what);
  if (a.experts < 1 || a.experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [1, %d]", what, MUON_MAX_EXPERTS);
  if (a.stride < a.experts || a.stride > kMaxStride)
    return fail(MUON_ERR_INVALID_ARG, "%s: logits_stride must be in [experts, 2^36]", what);
  if (!std::isfinite(a.coef)) return fail(MUON_ERR_INVALID_ARG, "%s: coef must be finite", what);
  return MUON_OK;
}
size_t balance_bytes(int64_t tokens, int32_t experts) {
  return align256((size_t)balance_blocks(tokens, experts) * (2 * experts + 1) * sizeof(float));
}

}  // namespace

extern "C" {

muon_status_t muon_layer_norm(int32_t dtype, int32_t w_dtype, int64_t rows, int64_t width, float eps,
                              const void* x, int64_t x_stride, const void* w, const void* bias, void* y,
                              float* mean, float* rstd, void* stream) {
  const char* what = "muon_layer_norm";
  NormArgs a{};
  a.dtype = dtype; a.w_dtype = w_dtype; a.rows = rows; a.width = width; a.eps = eps;
  a.x = x; a.x_stride = x_stride; a.w = w; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
  muon_status_t st = check_norm(what, a);
  if (st == MUON_OK) st = check_pitch(what, x_stride, width);
  if (st != MUON_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(MUON_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", what);
  if (rows > 0 && (!x || !y)) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((st = check_stream(what, stream)) != MUON_OK || rows == 0) return st;
  return cuda_status(what, launch_norm(a, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_layer_norm_workspace(int64_t rows, int64_t width, size_t* bytes) {
  const char* what = "muon_layer_norm_workspace";
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "%s: bytes is NULL", what);
  NormArgs a{};
  a.rows = rows;
  a.width = width;
  const muon_status_t st = check_norm(what, a);
  if (st == MUON_OK) *bytes = rows ? norm_bytes(rows, width) : 0;
  return st;
}

muon_status_t muon_layer_norm_backward(int32_t dtype, int32_t w_dtype, int64_t rows, int64_t width, const void* dy,
                                       int64_t dy_stride, const void* x, int64_t x_stride, const float* mean,
                                       const float* rstd, const void* w, const void* residual,
                                       int64_t residual_stride, void* dx, void* dw, void* db, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const char* what = "muon_layer_norm_backward";
  NormArgs a{};
  a.dtype = dtype; a.w_dtype = w_dtype; a.rows = rows; a.width = width;
  a.x = x; a.x_stride = x_stride; a.w = w;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.dy = dy; a.dy_stride = dy_stride; a.dx = dx; a.dw = dw; a.db = db;
  a.residual = residual; a.r_stride = residual ? residual_stride : 0;
  muon_status_t st = check_norm(what, a);
  if (st == MUON_OK) st = check_pitch(what, x_stride, width);
  if (st == MUON_OK) st = check_pitch(what, dy_stride, width);
  if (st == MUON_OK && residual) st = check_pitch(what, residual_stride, width);
  if (st != MUON_OK) return st;
  if (!dx && !dw && !db) return fail(MUON_ERR_INVALID_ARG, "%s: dx, dw and db are all NULL", what);
  if (rows > 0 && (!dy || !x || !mean || !rstd)) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const bool sums = dw || db;
  if (sums && rows > 0) st = check_workspace(what, workspace, workspace_bytes, norm_bytes(rows, width));
  if (st != MUON_OK || (st = check_stream(what, stream)) != MUON_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    cudaError_t e = cudaSuccess;
    const size_t bytes = (size_t)(width * dtype_size(w_dtype));
    if (dw) e = cudaMemsetAsync(dw, 0, bytes, s);
    if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, bytes, s);
    return cuda_status(what, e);
  }
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  return cuda_status(what, launch_norm_backward(a, s));
}

muon_status_t muon_balance_loss_workspace(int64_t tokens, int32_t experts, size_t* bytes) {
  const char* what = "muon_balance_loss_workspace";
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "%s: bytes is NULL", what);
  BalanceArgs a{};
  a.tokens = tokens;
  a.experts = experts;
  a.stride = experts;
  const muon_status_t st = check_balance(what, a);
  if (st == MUON_OK) *bytes = balance_bytes(tokens, experts);
  return st;
}

muon_status_t muon_balance_loss(int32_t dtype, int64_t tokens, int32_t experts, int32_t top_k, float coef,
                                const void* logits, int64_t logits_stride, const int32_t* indices, float* loss,
                                int32_t* counts, int32_t* live, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const char* what = "muon_balance_loss";
  BalanceArgs a{};
  a.dtype = dtype; a.tokens = tokens; a.experts = experts; a.top_k = top_k; a.coef = coef;
  a.logits = logits; a.stride = logits_stride; a.indices = indices;
  a.loss = loss; a.counts = counts; a.live = live;
  muon_status_t st = check_balance(what, a);
  if (st != MUON_OK) return st;
  if (top_k < 1 || top_k > experts || top_k > MUON_MAX_TOP_K)
    return fail(MUON_ERR_INVALID_ARG, "%s: top_k must be in [1, min(experts, %d)]", what, MUON_MAX_TOP_K);
  if (tokens * top_k > 0x7fffffffll) return fail(MUON_ERR_INVALID_ARG, "%s: tokens * top_k exceeds 2^31 - 1", what);
  if (!loss || !counts || !live || (tokens > 0 && (!logits || !indices)))
    return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  st = check_workspace(what, workspace, workspace_bytes, balance_bytes(tokens, experts));
  if (st == MUON_OK) st = check_stream(what, stream);
  if (st != MUON_OK) return st;
  a.blocks = balance_blocks(tokens, experts);
  a.part = static_cast<float*>(workspace);
  a.part_counts = reinterpret_cast<int32_t*>(a.part + (int64_t)a.blocks * experts);
  return cuda_status(what, launch_balance(a, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_balance_loss_backward(int32_t dtype, int64_t tokens, int32_t experts, float coef,
                                         const float* dloss, const void* logits, int64_t logits_stride,
                                         const int32_t* counts, const int32_t* live, const void* residual,
                                         int64_t residual_stride, void* dlogits, void* stream) {
  const char* what = "muon_balance_loss_backward";
  BalanceArgs a{};
  a.dtype = dtype; a.tokens = tokens; a.experts = experts; a.coef = coef;
  a.dloss = dloss; a.logits = logits; a.stride = logits_stride;
  a.counts = const_cast<int32_t*>(counts); a.live = const_cast<int32_t*>(live);
  a.residual = residual; a.r_stride = residual ? residual_stride : 0; a.dlogits = dlogits;
  muon_status_t st = check_balance(what, a);
  if (st == MUON_OK && residual) st = check_pitch(what, residual_stride, experts);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!dloss || !logits || !counts || !live || !dlogits))
    return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((st = check_stream(what, stream)) != MUON_OK || tokens == 0) return st;
  return cuda_status(what, launch_balance_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
