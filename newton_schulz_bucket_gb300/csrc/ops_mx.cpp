// Microscaled 4-bit weights and their products behind the C ABI
// (include/muon_ops.h): argument checks and launches.
#include "ops_checks.h"

using namespace muon;

namespace {

int64_t blocks_of(int64_t n) { return (n + 31) / 32; }

muon_status_t check_matrix(const char* what, int32_t dtype, int32_t experts, int64_t in, int64_t out) {
  if (!dtype_ok(dtype)) return fail(MUON_ERR_INVALID_ARG, "%s: dtype is not a muon_dtype_t", what);
  if (experts < 0 || experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [0, %d]", what, MUON_MAX_EXPERTS);
  if (in < 1 || in > kMaxDim || out < 1 || out > kMaxDim)
    return fail(MUON_ERR_INVALID_ARG, "%s: in and out must be in [1, 2^30]", what);
  return MUON_OK;
}
muon_status_t check_held(const char* what, const void* values, const void* scales) {
  if (!values || !scales) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (reinterpret_cast<uintptr_t>(values) & 15)
    return fail(MUON_ERR_INVALID_ARG, "%s: values must start on 16 bytes", what);
  return MUON_OK;
}
muon_status_t check_blocks(const char* what, int64_t rows, int64_t mat_rows, int64_t cols) {
  if (mx_blocks(rows, mat_rows, cols) > kMaxBlocks)
    return fail(MUON_ERR_UNSUPPORTED, "%s: too many blocks for one launch", what);
  return MUON_OK;
}

// The rounded token rows and both operands' ordered scales in the workspace.
struct Scratch {
  size_t x_scales, w_scales, total;
  int tile_rows;
};
Scratch scratch_of(const muon_mx_linear_args* a) {
  Scratch c{};
  const int64_t parts = mx_parts(a->in), mats = a->experts ? a->experts : 1;
  c.tile_rows = mx_tile_rows(a->rows, a->experts, a->out);
  if (a->rows == 0 || mx_own_rows(a->rows, a->experts)) return c;
  c.x_scales = align256((size_t)(a->rows * blocks_of(a->in) * 16));
  c.w_scales = c.x_scales + align256((size_t)(mx_token_slots(a->rows, a->experts, c.tile_rows) * parts * 512 *
                                              mx_token_blocks(c.tile_rows)));
  c.total = c.w_scales + align256((size_t)(mats * ((a->out + 127) / 128) * parts * 512));
  return c;
}

muon_status_t check_product(const char* what, const muon_mx_linear_args* a) {
  if (!a) return fail(MUON_ERR_INVALID_ARG, "%s: args is NULL", what);
  muon_status_t st = check_matrix(what, a->dtype, a->experts, a->in, a->out);
  if (st != MUON_OK) return st;
  if (a->activation < ACT_NONE || a->activation > ACT_GELU_TANH)
    return fail(MUON_ERR_INVALID_ARG, "%s: activation is not a muon_activation_t", what);
  if (a->rows < 0 || a->rows > kMaxDim) return fail(MUON_ERR_INVALID_ARG, "%s: rows must be in [0, 2^30]", what);
  if (a->x_stride < a->in || a->x_stride > kMaxStride)
    return fail(MUON_ERR_INVALID_ARG, "%s: x_stride must be in [in, 2^36]", what);
  if (a->residual && (a->residual_stride < a->out || a->residual_stride > kMaxStride))
    return fail(MUON_ERR_INVALID_ARG, "%s: residual_stride must be in [out, 2^36]", what);
  const int64_t mats = a->experts ? a->experts : 1;
  if ((a->rows / 64 + mats) * ((a->out + 255) / 256) > kMaxBlocks)
    return fail(MUON_ERR_UNSUPPORTED, "%s: too many tiles for one launch", what);
  // token rows' ordered scales are placed in words of 32 bits
  const int tile = mx_tile_rows(a->rows, a->experts, a->out);
  if (mx_token_slots(a->rows, a->experts, tile) * mx_parts(a->in) * mx_token_blocks(tile) >= (0xffffffffll >> 7))
    return fail(MUON_ERR_UNSUPPORTED, "%s: [%lld, %lld] has too many scales", what, (long long)a->rows, (long long)a->in);
  if (mx_prepare_blocks(a->rows, a->in, a->out, mats) > kMaxBlocks)
    return fail(MUON_ERR_UNSUPPORTED, "%s: too many blocks for one launch", what);
  return MUON_OK;
}

}  // namespace

extern "C" {

muon_status_t muon_mx_quantize(int32_t dtype, int32_t w_layout, int32_t experts, int64_t in, int64_t out,
                               const void* w, int64_t w_stride, int64_t w_expert_stride, void* values, void* scales,
                               void* stream) {
  const char* what = "muon_mx_quantize";
  muon_status_t st = check_matrix(what, dtype, experts, in, out);
  if (st != MUON_OK) return st;
  if (w_layout != MUON_W_IN_OUT && w_layout != MUON_W_OUT_IN)
    return fail(MUON_ERR_INVALID_ARG, "%s: w_layout is not a muon_weight_layout_t", what);
  const int64_t w_row = w_layout == MUON_W_IN_OUT ? out : in, w_rows = w_layout == MUON_W_IN_OUT ? in : out;
  if (w_stride < w_row || w_stride > kMaxStride)
    return fail(MUON_ERR_INVALID_ARG, "%s: w_stride must be in [a row's length, 2^36]", what);
  if (experts > 1 && (w_expert_stride > kMaxStride || w_expert_stride < w_row ||
                      (w_expert_stride - w_row) / w_stride < w_rows - 1))
    return fail(MUON_ERR_INVALID_ARG, "%s: w_expert_stride is shorter than one matrix, or exceeds 2^36", what);
  if (!w) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  MxRows q{};
  q.src = w;
  q.stride = w_stride;
  q.batch_stride = experts > 1 ? w_expert_stride : 0;
  q.mat_rows = out;
  q.rows = out * (experts ? experts : 1);
  q.cols = in;
  q.values = static_cast<uint8_t*>(values);
  q.scales = static_cast<uint8_t*>(scales);
  st = check_held(what, values, scales);
  if (st == MUON_OK) st = check_blocks(what, q.rows, q.mat_rows, in);
  if (st == MUON_OK) st = check_stream(what, stream);
  if (st != MUON_OK) return st;
  return cuda_status(what, launch_mx_rows(dtype, w_layout == MUON_W_IN_OUT ? MX_ACROSS : MX_ALONG, q,
                                          static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_mx_dequantize(int32_t dtype, int32_t experts, int64_t in, int64_t out, const void* values,
                                 const void* scales, void* w, void* stream) {
  const char* what = "muon_mx_dequantize";
  muon_status_t st = check_matrix(what, dtype, experts, in, out);
  if (st == MUON_OK) st = check_held(what, values, scales);
  if (st != MUON_OK) return st;
  if (!w) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  MxRows q{};
  q.mat_rows = out;
  q.rows = out * (experts ? experts : 1);
  q.cols = in;
  q.values = static_cast<uint8_t*>(const_cast<void*>(values));
  q.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  q.dst = w;
  st = check_blocks(what, q.rows, q.rows, in);
  if (st == MUON_OK) st = check_stream(what, stream);
  if (st != MUON_OK) return st;
  return cuda_status(what, launch_mx_rows(dtype, MX_BACK, q, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_mx_linear_workspace(const muon_mx_linear_args* args, size_t* bytes) {
  const char* what = "muon_mx_linear_workspace";
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "%s: bytes is NULL", what);
  const muon_status_t st = check_product(what, args);
  if (st == MUON_OK) *bytes = scratch_of(args).total;
  return st;
}

muon_status_t muon_mx_linear(const muon_mx_linear_args* args, void* stream) {
  const char* what = "muon_mx_linear";
  muon_status_t st = check_product(what, args);
  if (st != MUON_OK) return st;
  const muon_mx_linear_args& a = *args;
  st = check_held(what, a.w_values, a.w_scales);
  if (st != MUON_OK) return st;
  if (a.experts > 0 && !a.offsets) return fail(MUON_ERR_INVALID_ARG, "%s: offsets is NULL with experts > 0", what);
  if (a.rows > 0 && (!a.x || !a.y)) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const Scratch c = scratch_of(args);
  st = check_workspace(what, a.workspace, a.workspace_bytes, c.total);
  if (st == MUON_OK) st = check_stream(what, stream);
  if (st != MUON_OK || a.rows == 0) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  MxPrepare q{};
  q.x.src = a.x;
  q.x.stride = a.x_stride;
  q.x.rows = q.x.mat_rows = a.rows;
  q.x.cols = a.in;
  q.x.values = ws;
  q.x.scales = ws + c.x_scales;
  q.experts = a.experts; q.offsets = a.offsets; q.tile_rows = c.tile_rows;
  q.w_scales = static_cast<const uint8_t*>(a.w_scales);
  q.w_ordered = ws + c.w_scales;
  q.out = a.out;
  q.mats = a.experts ? a.experts : 1;
  MxProduct p{};
  p.dtype = a.dtype; p.act = a.activation; p.experts = a.experts; p.offsets = a.offsets; p.tile_rows = c.tile_rows;
  p.rows = a.rows; p.in = a.in; p.out = a.out;
  p.x_values = q.x.values; p.x_scales = q.x.scales;
  p.w_values = static_cast<const uint8_t*>(a.w_values);
  p.w_scales = q.w_ordered;
  p.bias = a.bias; p.residual = a.residual; p.r_stride = a.residual ? a.residual_stride : 0; p.y = a.y;
  const bool own = mx_own_rows(a.rows, a.experts);
  if (own) {
    p.x = a.x;
    p.x_stride = a.x_stride;
    p.w_scales = q.w_scales;
  }
  cudaError_t e = ops_error_word(&p.err);
  if (e == cudaSuccess && !own) e = launch_mx_prepare(a.dtype, q, s);
  if (e == cudaSuccess) e = launch_mx_linear(p, s);
  return cuda_status(what, e);
}

}  // extern "C"
