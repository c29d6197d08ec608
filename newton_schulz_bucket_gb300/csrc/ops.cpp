// The layer operators behind the C ABI (include/muon_ops.h): argument checks,
// the products a call is made of, and their launches.
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/muon_ops.h"
#include "internal.h"
#include "ops.h"

using namespace muon;

namespace {

muon_status_t fail(muon_status_t st, const char* fmt, ...) {
  char buf[320];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

muon_status_t cuda_status(const char* what, cudaError_t e) {
  return e == cudaSuccess ? MUON_OK : fail(MUON_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool dtype_ok(int32_t t) { return t == DT_F32 || t == DT_F16 || t == DT_BF16; }
int64_t dtype_size(int32_t t) { return t == DT_F32 ? 4 : 2; }

constexpr int64_t kMaxDim = 1ll << 30;
constexpr int64_t kMaxBlocks = 0x7fffffffll - 1024;  // (item counters run ahead by a grid's pairs)
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Launches go to the current device, so the stream has to be one of its own.
// A capturing stream cannot be asked (the query would end the capture).
muon_status_t check_stream(const char* what, void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (s == nullptr || s == cudaStreamLegacy || s == cudaStreamPerThread) return MUON_OK;
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capturing) == cudaSuccess && capturing != cudaStreamCaptureStatusNone) return MUON_OK;
  int dev = 0, sdev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MUON_ERR_CUDA, "%s: cudaGetDevice failed", what);
  if (cudaStreamGetDevice(s, &sdev) != cudaSuccess) {
    cudaGetLastError();  // not left for the next call to report
    return fail(MUON_ERR_INVALID_ARG, "%s: stream is not a valid CUDA stream", what);
  }
  if (sdev != dev)
    return fail(MUON_ERR_INVALID_ARG, "%s: stream belongs to another device than the current one", what);
  return MUON_OK;
}

// ---- linear ----

// Scratch of one call, carved from the workspace in order.
struct Carve {
  uint8_t* base;
  size_t used = 0;
  void* take(size_t bytes) {
    const size_t at = used;
    used += align256(bytes);
    return base ? base + at : nullptr;
  }
};

muon_status_t check_linear(const muon_linear_args* a, bool backward, const char* what) {
  if (!a) return fail(MUON_ERR_INVALID_ARG, "%s: args is NULL", what);
  if (!dtype_ok(a->dtype)) return fail(MUON_ERR_INVALID_ARG, "%s: dtype is not a muon_dtype_t", what);
  if (a->activation < ACT_NONE || a->activation > ACT_GELU_TANH)
    return fail(MUON_ERR_INVALID_ARG, "%s: activation is not a muon_activation_t", what);
  if (a->w_layout != MUON_W_IN_OUT && a->w_layout != MUON_W_OUT_IN)
    return fail(MUON_ERR_INVALID_ARG, "%s: w_layout is not a muon_weight_layout_t", what);
  if (a->experts < 0 || a->experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [0, %d]", what, MUON_MAX_EXPERTS);
  if (a->rows < 0 || a->rows > kMaxDim || a->in < 1 || a->in > kMaxDim || a->out < 1 || a->out > kMaxDim)
    return fail(MUON_ERR_INVALID_ARG, "%s: rows must be in [0, 2^30], in and out in [1, 2^30]", what);
  const int64_t w_row = a->w_layout == MUON_W_IN_OUT ? a->out : a->in;
  const int64_t w_rows = a->w_layout == MUON_W_IN_OUT ? a->in : a->out;
  if (a->x_stride < a->in || a->w_stride < w_row)
    return fail(MUON_ERR_INVALID_ARG, "%s: a row stride is shorter than its row", what);
  if (a->x_stride > (1ll << 36) || a->w_stride > (1ll << 36) || a->w_expert_stride > (1ll << 36) ||
      a->residual_stride > (1ll << 36) || a->dy_stride > (1ll << 36))
    return fail(MUON_ERR_INVALID_ARG, "%s: a stride exceeds 2^36 elements", what);
  if (a->experts > 1 && (a->w_expert_stride < w_row || (a->w_expert_stride - w_row) / a->w_stride < w_rows - 1))
    return fail(MUON_ERR_INVALID_ARG, "%s: w_expert_stride is shorter than one matrix", what);
  if (a->experts > 0 && !a->offsets)
    return fail(MUON_ERR_INVALID_ARG, "%s: offsets is NULL with experts > 0", what);
  // what the kernels count in 32 bits, in the smallest tiles that tile_plan may take
  const auto up = [](int64_t v, int64_t by) { return (v + by - 1) / by; };
  const int64_t mats = a->experts ? a->experts : 1, wide = a->in > a->out ? a->in : a->out;
  const int64_t narrow = a->in > a->out ? a->out : a->in, row_blocks = up(a->rows, 4) * up(wide, 2048);
  const int64_t counts[] = {
      (up(a->rows, 64) + mats) * up(wide, 256) * 16,                     // rows form: token tiles x features x parts
      up(wide, 128) * up(narrow, 128),                                   // sum form: a matrix's tiles
      2 * row_blocks, row_blocks + mats * up(w_rows, 4) * up(w_row, 2048),  // operands padded or split, two a launch
      up(a->rows, 128) * up(a->out, 32), up(a->out, 256) * mats,         // the gradient's first pass
      up(a->rows * wide, 256), up(narrow * wide, 256)};                  // the join of a split sum
  for (const int64_t n : counts)
    if (n > kMaxBlocks)
      return fail(MUON_ERR_UNSUPPORTED, "%s: [%lld, %lld] x [%lld, %lld] with %d experts has too many tiles", what,
                  (long long)a->rows, (long long)a->in, (long long)a->in, (long long)a->out, a->experts);
  if (!backward) {
    if (!a->w || (a->rows > 0 && (!a->x || !a->y)))
      return fail(MUON_ERR_INVALID_ARG, "%s: x, w and y must be non-NULL", what);
    if (a->residual && a->residual_stride < a->out)
      return fail(MUON_ERR_INVALID_ARG, "%s: a row stride is shorter than its row", what);
  } else {
    if (!a->dx && !a->dw && !a->db)
      return fail(MUON_ERR_INVALID_ARG, "%s: dx, dw and db are all NULL", what);
    if (a->rows > 0 && (!a->dy || (a->dx && !a->w) || (a->dw && !a->x) || (a->activation != ACT_NONE && !a->preact)))
      return fail(MUON_ERR_INVALID_ARG, "%s: dy, x, w and (with an activation) preact must be non-NULL", what);
    if (a->dy_stride < a->out)
      return fail(MUON_ERR_INVALID_ARG, "%s: a row stride is shorter than its row", what);
  }
  return MUON_OK;
}

Product forward_product(const muon_linear_args* a) {
  Product p{};
  p.dtype = a->dtype;
  p.mode = a->experts ? GROUP_ROWS : GROUP_NONE;
  p.experts = a->experts;
  p.offsets = a->offsets;
  p.M = a->rows; p.N = a->out; p.K = a->in;
  p.A = a->x; p.a_m = a->x_stride; p.a_k = 1;
  p.B = a->w;
  p.b_k = a->w_layout == MUON_W_IN_OUT ? a->w_stride : 1;
  p.b_n = a->w_layout == MUON_W_IN_OUT ? 1 : a->w_stride;
  p.b_e = a->w_expert_stride;
  p.D = a->y;
  p.act = a->activation;
  p.bias = a->bias;
  p.residual = a->residual; p.r_m = a->residual_stride;
  p.preact = a->preact_out;
  return p;
}

// dx = dz W^T
Product dx_product(const muon_linear_args* a, const void* dz, int64_t dz_stride) {
  Product p{};
  p.dtype = a->dtype;
  p.mode = a->experts ? GROUP_ROWS : GROUP_NONE;
  p.experts = a->experts;
  p.offsets = a->offsets;
  p.M = a->rows; p.N = a->in; p.K = a->out;
  p.A = dz; p.a_m = dz_stride; p.a_k = 1;
  p.B = a->w;
  p.b_k = a->w_layout == MUON_W_IN_OUT ? 1 : a->w_stride;
  p.b_n = a->w_layout == MUON_W_IN_OUT ? a->w_stride : 1;
  p.b_e = a->w_expert_stride;
  p.D = a->dx;
  return p;
}

// dw = x^T dz, or for OUT_IN its transpose dz^T x
Product dw_product(const muon_linear_args* a, const void* x, int64_t x_stride, const void* dz, int64_t dz_stride) {
  Product p{};
  p.dtype = a->dtype;
  p.mode = a->experts ? GROUP_SUM : GROUP_NONE;
  p.experts = a->experts;
  p.offsets = a->offsets;
  p.K = a->rows;
  const bool io = a->w_layout == MUON_W_IN_OUT;
  p.M = io ? a->in : a->out;
  p.N = io ? a->out : a->in;
  p.A = io ? x : dz; p.a_m = 1; p.a_k = io ? x_stride : dz_stride;
  p.B = io ? dz : x; p.b_k = io ? dz_stride : x_stride; p.b_n = 1;
  p.D = a->dw;
  return p;
}

// An operand of the tensor-core form.  16-bit types: as it is where TMA can read
// it (base and row pitch multiples of 16 bytes), else a copy with padded rows in
// scratch.  fp32: its three bf16 planes in scratch.  (r, c) strides of the
// operand are (stride, 1) over rows x cols, batch apart.
struct Operand {
  const void* p;
  int64_t stride, batch_stride;
};
// `waiting` holds a job that has not been launched: two go together.
Operand tma_operand(int32_t dtype, Operand o, int64_t rows, int64_t cols, int64_t batch, Carve& c, bool launch,
                    RowsJob* waiting, cudaStream_t s, cudaError_t* e, const int32_t* offsets = nullptr) {
  const bool split = dtype == DT_F32;
  if (rows == 1 && batch == 1 && !split) o.stride = (o.stride + 7) / 8 * 8;  // no second row: any pitch does
  const bool ok = !split && (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && o.stride % 8 == 0 &&
                  (batch == 1 || o.batch_stride % 8 == 0);
  if (ok) return o;
  const int64_t pitch = (cols + 7) / 8 * 8;
  void* dst = c.take((size_t)(batch * (split ? 3 : 1) * rows * pitch * 2));
  const RowsJob mine{o.p, o.stride, o.batch_stride, static_cast<uint16_t*>(dst), pitch, rows, cols, batch,
                     offsets};
  if (waiting->batch == 0) {
    *waiting = mine;
  } else {
    if (launch && *e == cudaSuccess) *e = launch_prepare_rows(split, *waiting, mine, s);
    *waiting = RowsJob{};
  }
  return {dst, pitch, rows * pitch};
}

// One product.  `ready` operands went through tma_operand already.
cudaError_t run_product(Product p, bool a_ready, bool b_ready, Carve& c, bool launch, RowsJob waiting,
                        cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool a_along = p.a_k == 1, b_along = p.b_k == 1;
  const int64_t mats = p.mode == GROUP_ROWS ? p.experts : 1;
  if (!a_ready) {
    const Operand a = tma_operand(p.dtype, {p.A, a_along ? p.a_m : p.a_k, 0}, a_along ? p.M : p.K,
                                  a_along ? p.K : p.M, 1, c, launch, &waiting, s, &e);
    p.A = a.p;
    (a_along ? p.a_m : p.a_k) = a.stride;
  }
  if (!b_ready) {
    const Operand b = tma_operand(p.dtype, {p.B, b_along ? p.b_n : p.b_k, p.b_e}, b_along ? p.N : p.K,
                                  b_along ? p.K : p.N, mats, c, launch, &waiting, s, &e,
                                  p.mode == GROUP_ROWS ? p.offsets : nullptr);
    p.B = b.p;
    (b_along ? p.b_n : p.b_k) = b.stride;
    p.b_e = b.batch_stride;
  }
  if (launch && e == cudaSuccess && waiting.batch) e = launch_prepare_rows(p.dtype == DT_F32, waiting, RowsJob{}, s);
  if (linear_few_fits(p)) {
    if (!launch || e != cudaSuccess) return e;
    e = ops_error_word(&p.err);
    return e == cudaSuccess ? launch_linear_few(p, s) : e;
  }
  const TilePlan t = tile_plan(p);
  float* part = t.part_bytes ? static_cast<float*>(c.take((size_t)t.part_bytes)) : nullptr;
  if (!launch || e != cudaSuccess) return e;
  e = ops_error_word(&p.err);
  return e == cudaSuccess ? launch_linear_tc(p, t, part, s) : e;
}

muon_status_t run_linear(const muon_linear_args* a, bool backward, Carve& c, bool launch, cudaStream_t s) {
  if (!backward) {
    if (a->rows == 0) return MUON_OK;
    return cuda_status("muon_linear", run_product(forward_product(a), false, false, c, launch, RowsJob{}, s));
  }
  const char* what = "muon_linear_backward";
  const int64_t b = dtype_size(a->dtype);
  const int64_t mats = a->experts ? a->experts : 1;
  if (a->rows == 0) {
    cudaError_t e = cudaSuccess;
    if (launch && a->dw) e = cudaMemsetAsync(a->dw, 0, (size_t)(mats * a->in * a->out * b), s);
    if (launch && a->db && e == cudaSuccess) e = cudaMemsetAsync(a->db, 0, (size_t)(mats * a->out * b), s);
    return cuda_status(what, e);
  }
  const bool act = a->activation != ACT_NONE, products = a->dx || a->dw;
  GradPrep g{};
  g.dtype = a->dtype; g.act = a->activation; g.experts = a->experts; g.offsets = a->offsets;
  g.rows = a->rows; g.cols = a->out;
  g.dy = a->dy; g.dy_stride = a->dy_stride; g.z = a->preact;
  g.db = a->db;
  g.dz_stride = (a->out + 7) / 8 * 8;
  if (act && products) g.dz = c.take((size_t)(a->rows * g.dz_stride * b));
  if (a->db && a->rows > kGradSingle)
    g.part = static_cast<float*>(c.take(((a->rows + kGradChunk - 1) / kGradChunk + mats) * a->out * sizeof(float)));
  cudaError_t e = cudaSuccess;
  if (launch && (act || a->db)) e = launch_grad_prep(g, s);
  Operand dz{act ? g.dz : a->dy, act ? g.dz_stride : a->dy_stride, 0};
  Operand x{a->x, a->x_stride, 0};
  RowsJob waiting{};
  if (products) dz = tma_operand(a->dtype, dz, a->rows, a->out, 1, c, launch, &waiting, s, &e);  // once for both
  if (a->dw) x = tma_operand(a->dtype, x, a->rows, a->in, 1, c, launch, &waiting, s, &e);
  if (a->dx && e == cudaSuccess) {
    e = run_product(dx_product(a, dz.p, dz.stride), true, false, c, launch, waiting, s);
    waiting = RowsJob{};
  }
  if (a->dw && e == cudaSuccess)
    e = run_product(dw_product(a, x.p, x.stride, dz.p, dz.stride), true, true, c, launch, waiting, s);
  return cuda_status(what, e);
}

muon_status_t linear_entry(const muon_linear_args* a, bool backward, void* stream) {
  const char* what = backward ? "muon_linear_backward" : "muon_linear";
  muon_status_t st = check_linear(a, backward, what);
  if (st == MUON_OK) st = check_stream(what, stream);
  if (st != MUON_OK) return st;
  Carve sizes{nullptr};
  st = run_linear(a, backward, sizes, false, nullptr);
  if (st != MUON_OK) return st;
  if (sizes.used > 0 && (!a->workspace || a->workspace_bytes < sizes.used ||
                         (reinterpret_cast<uintptr_t>(a->workspace) & 255) != 0))
    return fail(MUON_ERR_INVALID_ARG, "%s: needs a 256-byte aligned workspace of %zu bytes", what, sizes.used);
  Carve c{static_cast<uint8_t*>(a->workspace)};
  return run_linear(a, backward, c, true, static_cast<cudaStream_t>(stream));
}

// ---- gate ----

muon_status_t check_gate(const char* what, const GateArgs& g, bool backward, void* stream) {
  if (!dtype_ok(g.dtype)) return fail(MUON_ERR_INVALID_ARG, "%s: dtype is not a muon_dtype_t", what);
  if (g.tokens < 0 || g.tokens > kMaxDim) return fail(MUON_ERR_INVALID_ARG, "%s: tokens must be in [0, 2^30]", what);
  if (g.experts < 1 || g.experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [1, %d]", what, MUON_MAX_EXPERTS);
  if (g.top_k < 1 || g.top_k > g.experts || g.top_k > MUON_MAX_TOP_K)
    return fail(MUON_ERR_INVALID_ARG, "%s: top_k must be in [1, min(experts, %d)]", what, MUON_MAX_TOP_K);
  if (g.stride < g.experts || g.stride > (1ll << 36))
    return fail(MUON_ERR_INVALID_ARG, "%s: logits_stride must be in [experts, 2^36]", what);
  if (g.tokens > 0 && (!g.logits || !g.indices || (backward ? !g.dweights || !g.dlogits : !g.weights)))
    return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  return check_stream(what, stream);
}

// ---- sort ----

muon_status_t check_rows(const char* what, int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k) {
  if (!dtype_ok(dtype)) return fail(MUON_ERR_INVALID_ARG, "%s: dtype is not a muon_dtype_t", what);
  if (top_k < 1 || top_k > MUON_MAX_TOP_K)
    return fail(MUON_ERR_INVALID_ARG, "%s: top_k must be in [1, %d]", what, MUON_MAX_TOP_K);
  if (tokens < 0 || tokens > kMaxDim || tokens * top_k > 0x7fffffffll - kSortChunk)
    return fail(MUON_ERR_INVALID_ARG, "%s: tokens * top_k must be in [0, 2^31 - 1025]", what);
  if (hidden < 1 || hidden > kMaxDim) return fail(MUON_ERR_INVALID_ARG, "%s: hidden must be in [1, 2^30]", what);
  return MUON_OK;
}

muon_status_t check_row_stride(const char* what, int64_t stride, int64_t hidden) {
  if (stride < hidden || stride > (1ll << 36))
    return fail(MUON_ERR_INVALID_ARG, "%s: a row stride must be in [hidden, 2^36]", what);
  return MUON_OK;
}

size_t dispatch_bytes(int64_t tokens, int32_t top_k, int32_t experts) {
  if (tokens * top_k <= kSortCluster) return 0;
  const size_t chunks = (size_t)((tokens * top_k + kSortChunk - 1) / kSortChunk);
  return align256((chunks + 1) * experts * sizeof(int32_t));
}

}  // namespace

extern "C" {

muon_status_t muon_linear_workspace(const muon_linear_args* args, int32_t backward, size_t* bytes) {
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "muon_linear_workspace: bytes is NULL");
  const muon_status_t st = check_linear(args, backward != 0, "muon_linear_workspace");
  if (st != MUON_OK) return st;
  Carve c{nullptr};
  const muon_status_t r = run_linear(args, backward != 0, c, false, nullptr);
  *bytes = c.used;
  return r;
}

muon_status_t muon_linear(const muon_linear_args* args, void* stream) {
  return linear_entry(args, false, stream);
}

muon_status_t muon_linear_backward(const muon_linear_args* args, void* stream) {
  return linear_entry(args, true, stream);
}

muon_status_t muon_gate(int32_t dtype, int64_t tokens, int32_t experts, int32_t top_k,
                        int32_t renormalize, const void* logits, int64_t logits_stride,
                        int32_t* indices, float* weights, void* stream) {
  GateArgs g{dtype, experts, top_k, renormalize != 0, tokens, logits_stride, logits, indices, weights,
             nullptr, nullptr};
  const muon_status_t st = check_gate("muon_gate", g, false, stream);
  if (st != MUON_OK || tokens == 0) return st;
  return cuda_status("muon_gate", launch_gate(g, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_gate_backward(int32_t dtype, int64_t tokens, int32_t experts, int32_t top_k,
                                 int32_t renormalize, const float* dweights, const void* logits,
                                 int64_t logits_stride, const int32_t* indices, void* dlogits,
                                 void* stream) {
  GateArgs g{dtype, experts, top_k, renormalize != 0, tokens, logits_stride, logits,
             const_cast<int32_t*>(indices), nullptr, dweights, dlogits};
  const muon_status_t st = check_gate("muon_gate_backward", g, true, stream);
  if (st != MUON_OK || tokens == 0) return st;
  return cuda_status("muon_gate_backward", launch_gate_backward(g, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_dispatch_workspace(int64_t tokens, int32_t top_k, int32_t experts, size_t* bytes) {
  const char* what = "muon_dispatch_workspace";
  if (!bytes) return fail(MUON_ERR_INVALID_ARG, "%s: bytes is NULL", what);
  const muon_status_t st = check_rows(what, DT_F32, tokens, 1, top_k);
  if (st != MUON_OK) return st;
  if (experts < 1 || experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [1, %d]", what, MUON_MAX_EXPERTS);
  *bytes = dispatch_bytes(tokens, top_k, experts);
  return MUON_OK;
}

muon_status_t muon_dispatch(int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k,
                            int32_t experts, const void* x, int64_t x_stride, const void* indices,
                            int32_t index_bits, void* xs, int32_t* slot, int32_t* offsets,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const char* what = "muon_dispatch";
  muon_status_t st = check_rows(what, dtype, tokens, hidden, top_k);
  if (st != MUON_OK) return st;
  if (experts < 1 || experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [1, %d]", what, MUON_MAX_EXPERTS);
  if (index_bits != 32 && index_bits != 64)
    return fail(MUON_ERR_INVALID_ARG, "%s: index_bits must be 32 or 64", what);
  if (xs && (st = check_row_stride(what, x_stride, hidden)) != MUON_OK) return st;
  if (!offsets || (tokens > 0 && (!indices || !slot || (xs && !x))))
    return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  const size_t need = dispatch_bytes(tokens, top_k, experts);
  if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0))
    return fail(MUON_ERR_INVALID_ARG, "%s: needs a 256-byte aligned workspace of %zu bytes", what, need);
  if ((st = check_stream(what, stream)) != MUON_OK) return st;
  SortArgs a{};
  a.dtype = dtype; a.top_k = top_k; a.experts = experts; a.index_bits = index_bits;
  a.tokens = tokens; a.hidden = hidden;
  a.x = x; a.x_stride = x_stride; a.indices = indices; a.xs = xs; a.slot = slot; a.offsets = offsets;
  a.counts = static_cast<int32_t*>(workspace);
  return cuda_status(what, launch_dispatch(a, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_dispatch_backward(int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k,
                                     const void* dxs, int64_t dxs_stride, const int32_t* slot,
                                     void* dx, void* stream) {
  const char* what = "muon_dispatch_backward";
  muon_status_t st = check_rows(what, dtype, tokens, hidden, top_k);
  if (st == MUON_OK) st = check_row_stride(what, dxs_stride, hidden);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!dxs || !slot || !dx)) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((st = check_stream(what, stream)) != MUON_OK || tokens == 0) return st;
  SortArgs a{};
  a.dtype = dtype; a.top_k = top_k; a.tokens = tokens; a.hidden = hidden;
  a.ys = dxs; a.ys_stride = dxs_stride; a.slot = const_cast<int32_t*>(slot); a.y = dx;
  return cuda_status(what, launch_combine(a, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_combine(int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k,
                           const void* ys, int64_t ys_stride, const int32_t* slot,
                           const float* weights, const void* residual, int64_t residual_stride,
                           void* y, void* stream) {
  const char* what = "muon_combine";
  muon_status_t st = check_rows(what, dtype, tokens, hidden, top_k);
  if (st == MUON_OK) st = check_row_stride(what, ys_stride, hidden);
  if (st == MUON_OK && residual) st = check_row_stride(what, residual_stride, hidden);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!ys || !slot || !weights || !y)) return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((st = check_stream(what, stream)) != MUON_OK || tokens == 0) return st;
  SortArgs a{};
  a.dtype = dtype; a.top_k = top_k; a.tokens = tokens; a.hidden = hidden;
  a.ys = ys; a.ys_stride = ys_stride; a.slot = const_cast<int32_t*>(slot); a.weights = weights;
  a.residual = residual; a.r_stride = residual ? residual_stride : 0; a.y = y;
  return cuda_status(what, launch_combine(a, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_combine_backward(int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k,
                                    int32_t experts, const void* dy, int64_t dy_stride,
                                    const void* ys, int64_t ys_stride, const int32_t* slot,
                                    const int32_t* offsets, const float* weights, void* dys,
                                    float* dweights, void* stream) {
  const char* what = "muon_combine_backward";
  muon_status_t st = check_rows(what, dtype, tokens, hidden, top_k);
  if (st == MUON_OK) st = check_row_stride(what, dy_stride, hidden);
  if (st == MUON_OK) st = check_row_stride(what, ys_stride, hidden);
  if (st != MUON_OK) return st;
  if (experts < 1 || experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "%s: experts must be in [1, %d]", what, MUON_MAX_EXPERTS);
  if (tokens > 0 && (!dy || !ys || !slot || !offsets || !weights || !dys || !dweights))
    return fail(MUON_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((st = check_stream(what, stream)) != MUON_OK || tokens == 0) return st;
  SortArgs a{};
  a.dtype = dtype; a.top_k = top_k; a.experts = experts; a.tokens = tokens; a.hidden = hidden;
  a.dy = dy; a.dy_stride = dy_stride; a.ys = ys; a.ys_stride = ys_stride;
  a.slot = const_cast<int32_t*>(slot); a.offsets = const_cast<int32_t*>(offsets);
  a.weights = weights; a.dys = dys; a.dweights = dweights;
  return cuda_status(what, launch_combine_backward(a, static_cast<cudaStream_t>(stream)));
}

muon_status_t muon_ops_check_error(void) {
  const char* what = "muon_ops_check_error";
  int* err = nullptr;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = ops_error_word(&err);
  int word = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && word) e = cudaMemset(err, 0, sizeof word);
  if (e != cudaSuccess) return cuda_status(what, e);
  return word ? fail(MUON_ERR_TIMEOUT, "%s: a bounded wait ran out in an earlier call (code %d)", what, word) : MUON_OK;
}

}  // extern "C"
