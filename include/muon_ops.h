/*
 * muon_ops.h -- C ABI of the layer operators that stand next to the Muon
 * update on one GB300 (sm_103a): the products of the layers whose weight
 * matrices and expert tensors muon_step updates, and the routing that feeds an
 * expert tensor.
 *
 *   linear            z = x W + b,  y = act(z) + r            one [in, out] matrix
 *   linear, experts   the same, row s with the matrix of the expert it is sorted to
 *   gate              the top-k experts of each token and their softmax weights
 *   dispatch          token rows copied into expert order
 *   combine           y[t] = sum_j weight[t, j] * ys[slot[t, j]] + r[t]
 *   layer norm        y = (x - mean) / sqrt(var + eps) * w + b, row by row
 *   balance loss      the load of a router's experts and the loss that evens it out
 * and the gradient of each; and for serving
 *   mx weights        matrices in microscaled 4-bit numbers, and back
 *   mx linear         linear with such weights, one matrix or an expert tensor
 *
 * Conventions, beyond those of muon.h (statuses, muon_last_error, streams):
 *  - Stateless calls.  Every buffer is the caller's; scratch is a caller
 *    buffer whose size the operator's _workspace call gives, 256-byte
 *    aligned, free for reuse once the call's work on `stream` is done.  No
 *    call allocates device memory or synchronises, so every call can
 *    be captured in a CUDA graph (the first call of each operator on a device
 *    sets kernel attributes: host work, make it before a capture).
 *  - The current device must be the device of `stream` and of the buffers.
 *  - Matrices are row-major; a *_stride is the distance between rows in
 *    elements (>= the row's length).  Outputs are contiguous unless said.
 *  - Inputs and outputs must not overlap.  Elements need only the alignment
 *    of their type: buffers whose base and strides are multiples of 16 bytes
 *    take the fastest loads.
 *  - Counts may be zero (rows, tokens); widths and top_k are at least 1.
 *  - Sums, softmax terms and activations are computed in fp32 and rounded once
 *    where they are stored, except that the backward pass rounds
 *    dz = dy * act'(z) to the operand type before its two products in the
 *    16-bit types.  Results do not depend on timing: the same call on the
 *    same inputs gives the same bits.
 *  - Waits inside kernels are bounded: one that runs out ends its kernel, and
 *    muon_ops_check_error reports it.
 */
#ifndef MUON_GB300_OPS_H
#define MUON_GB300_OPS_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MUON_DTYPE_F32 = 0, MUON_DTYPE_F16 = 1, MUON_DTYPE_BF16 = 2 } muon_dtype_t;

/* act(z): z; max(z, 0); z / (1 + e^-z); z (1 + erf(z / sqrt 2)) / 2;
 * z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2.  The slope of RELU at 0 is 0. */
typedef enum {
  MUON_ACT_NONE = 0,
  MUON_ACT_RELU = 1,
  MUON_ACT_SILU = 2,
  MUON_ACT_GELU = 3,
  MUON_ACT_GELU_TANH = 4
} muon_activation_t;

/* Storage of one weight matrix: IN_OUT is [in][out], OUT_IN is [out][in].
 * Weight gradients come in the same order, contiguous. */
typedef enum { MUON_W_IN_OUT = 0, MUON_W_OUT_IN = 1 } muon_weight_layout_t;

/* Most experts of an expert tensor and of a gate; most experts of a token. */
#define MUON_MAX_EXPERTS 1024
#define MUON_MAX_TOP_K 32

/* One product with its epilogue, or its gradient.
 *
 * experts = 0: one matrix.  experts = E >= 1: w is [E] matrices, and rows
 * offsets[e] .. offsets[e + 1] - 1 of x (device int32 [E + 1], not decreasing)
 * go through matrix e, with row e of bias [E, out].  Rows before offsets[0] and
 * from offsets[E] on belong to no expert: their outputs are zero and they add to
 * no gradient.
 * (Offsets outside [0, rows] are clamped, so they cannot lead out of a buffer; where they
 * decrease, rows get results of no meaning, and no access leads out of a buffer either.)
 *
 * muon_linear reads x, w, bias (nullable), residual (nullable; added after
 * the activation) and writes y, and z to preact_out (nullable) for the way
 * back.  muon_linear_backward reads dy, x, w and, unless activation is NONE,
 * preact, and writes those of dx, dw and db that are not NULL:
 *   dz = dy * act'(z), dx = dz W^T, dw = x^T dz, db = sum over rows of dz
 * (the residual's gradient is dy itself).  All tensors are of `dtype`.  fp32
 * operands are cut into three bf16 numbers that together hold their 24 bits (in
 * scratch), and six partial products summed in fp32 make a product to within
 * 2^-22 of its size (2^-24 is left out, the rest is the sum's rounding; a product
 * within 2^-7 of the largest number may come out infinite); below about 2^-100 an
 * operand loses low bits, and below 2^-134 it counts as zero.  Infinities and NaN
 * follow the formula. */
typedef struct {
  int32_t dtype;       /* muon_dtype_t                                        */
  int32_t activation;  /* muon_activation_t                                   */
  int32_t experts;     /* 0: one matrix; 1 .. MUON_MAX_EXPERTS                */
  int32_t w_layout;    /* muon_weight_layout_t                                */
  int64_t rows, in, out;
  int64_t x_stride;         /* row strides in elements                        */
  int64_t w_stride;         /* of one matrix as stored                        */
  int64_t w_expert_stride;  /* between matrices (experts > 0)                 */
  int64_t residual_stride;
  int64_t dy_stride;
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  const int32_t* offsets;
  const void* preact;       /* backward: z, contiguous [rows, out]            */
  const void* dy;
  void* y;
  void* preact_out;
  void* dx;                 /* contiguous [rows, in]                          */
  void* dw;                 /* contiguous, in w's layout                      */
  void* db;                 /* [out], or [experts, out]                       */
  void* workspace;
  size_t workspace_bytes;
} muon_linear_args;

/* Scratch bytes muon_linear (backward = 0) or muon_linear_backward (1) needs
 * for these arguments (pointers' alignment included; the workspace fields are
 * not read).  Errors: INVALID_ARG as the call itself. */
MUON_API muon_status_t muon_linear_workspace(const muon_linear_args* args, int32_t backward,
                                             size_t* bytes);

/* y = act(x W + b) + residual.  Errors, before any launch: INVALID_ARG (NULL
 * args, x, w or y with rows > 0, offsets NULL with experts > 0; a size, enum or
 * stride out of range; workspace too small or not 256-byte aligned; a stream
 * of another device), UNSUPPORTED (a launch of more than 2^31 - 1025 tiles or
 * blocks), CUDA. */
MUON_API muon_status_t muon_linear(const muon_linear_args* args, void* stream);

/* The gradients (above).  Errors: as muon_linear; also INVALID_ARG where dy, or
 * preact with an activation, is NULL, or dx, dw and db all are. */
MUON_API muon_status_t muon_linear_backward(const muon_linear_args* args, void* stream);

/* The gate: for each token the top_k experts with the largest logits, in
 * falling order, ties to the lower expert, and their weights, softmax over all
 * experts (renormalize = 0) or over the chosen ones (1).  A logit of -inf
 * masks its expert: a token with fewer than top_k open experts gets index -1
 * and weight 0 in the places left over (dispatch drops those).  A NaN logit is
 * not chosen either, and makes the weights of the token's chosen experts NaN.
 * logits: `dtype` [tokens, experts] with row stride logits_stride;
 * indices: int32 [tokens, top_k]; weights: fp32 [tokens, top_k].  Errors:
 * INVALID_ARG (NULL pointers with tokens > 0; experts not in [1,
 * MUON_MAX_EXPERTS]; top_k not in [1, min(experts, MUON_MAX_TOP_K)]; stride;
 * dtype; stream), CUDA. */
MUON_API muon_status_t muon_gate(int32_t dtype, int64_t tokens, int32_t experts, int32_t top_k,
                                 int32_t renormalize, const void* logits, int64_t logits_stride,
                                 int32_t* indices, float* weights, void* stream);

/* The gate's gradient, the choice held fixed: with p the softmax over all
 * experts (over the chosen ones if renormalize) and g the weights' gradient
 * spread to the chosen experts, dlogits = p * (g - <p, g>).  A masked expert
 * and a token with no expert get 0.  dlogits: `dtype`, contiguous.  Errors: as
 * muon_gate. */
MUON_API muon_status_t muon_gate_backward(int32_t dtype, int64_t tokens, int32_t experts,
                                          int32_t top_k, int32_t renormalize,
                                          const float* dweights, const void* logits,
                                          int64_t logits_stride, const int32_t* indices,
                                          void* dlogits, void* stream);

/* Scratch bytes of muon_dispatch. */
MUON_API muon_status_t muon_dispatch_workspace(int64_t tokens, int32_t top_k, int32_t experts,
                                               size_t* bytes);

/* Tokens into expert order.  Assignment (t, j) goes to row slot[t, j] of xs:
 * assignments are sorted by expert, within an expert by t, then j; an index
 * outside [0, experts) drops its assignment (slot -1).  Expert e owns rows
 * offsets[e] .. offsets[e + 1] - 1; xs has tokens * top_k rows, those from
 * offsets[experts] on are zero.  indices: int32 or int64 (index_bits 32 or
 * 64) [tokens, top_k] contiguous.  xs and slot and offsets are written; xs may
 * be NULL (the order alone; x is then not read).  Errors: INVALID_ARG (NULL
 * pointers, sizes, tokens * top_k > 2^31 - 1025, dtype, workspace, stream), CUDA. */
MUON_API muon_status_t muon_dispatch(int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k,
                                     int32_t experts, const void* x, int64_t x_stride,
                                     const void* indices, int32_t index_bits, void* xs,
                                     int32_t* slot, int32_t* offsets, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* dx[t] = sum_j dxs[slot[t, j]], j in order, over the slots that are not -1.
 * dxs: [tokens * top_k, hidden] with row stride dxs_stride; slots outside
 * that range count as -1.  Errors: INVALID_ARG, CUDA. */
MUON_API muon_status_t muon_dispatch_backward(int32_t dtype, int64_t tokens, int64_t hidden,
                                              int32_t top_k, const void* dxs, int64_t dxs_stride,
                                              const int32_t* slot, void* dx, void* stream);

/* y[t] = sum_j weights[t, j] * ys[slot[t, j]] + residual[t] (residual nullable),
 * j in order, over the slots that are not -1.  weights: fp32 [tokens, top_k].
 * Errors: INVALID_ARG, CUDA. */
MUON_API muon_status_t muon_combine(int32_t dtype, int64_t tokens, int64_t hidden, int32_t top_k,
                                    const void* ys, int64_t ys_stride, const int32_t* slot,
                                    const float* weights, const void* residual,
                                    int64_t residual_stride, void* y, void* stream);

/* dys[slot[t, j]] = weights[t, j] * dy[t] and dweights[t, j] = <ys[slot[t, j]],
 * dy[t]> (fp32; 0 for slot -1).  Rows of dys from offsets[experts] on are zero.
 * Errors: INVALID_ARG, CUDA. */
MUON_API muon_status_t muon_combine_backward(int32_t dtype, int64_t tokens, int64_t hidden,
                                             int32_t top_k, int32_t experts, const void* dy,
                                             int64_t dy_stride, const void* ys, int64_t ys_stride,
                                             const int32_t* slot, const int32_t* offsets,
                                             const float* weights, void* dys, float* dweights,
                                             void* stream);

/* Layer norm of each row: with mean and var (of width, not width - 1) of row t,
 * rstd = 1 / sqrt(var + eps),
 *   y[t] = (x[t] - mean[t]) * rstd[t] * w + bias.
 * x: `dtype` [rows, width] with row stride x_stride; w and bias: w_dtype (dtype or
 * F32) [width], nullable (ones, zeros); y: `dtype` [rows, width]; mean and rstd: fp32
 * [rows], nullable, for the way back.  The sums are fp32, as long as a row may be: one
 * whose elements add up beyond the largest fp32 number gets a mean of infinity, and one
 * whose squared deviations do an rstd of 0.  Errors: INVALID_ARG (NULL x or y with rows >
 * 0; rows not in [0, 2^30], width not in [1, 2^30]; eps negative or not finite;
 * stride; dtypes; stream), CUDA. */
MUON_API muon_status_t muon_layer_norm(int32_t dtype, int32_t w_dtype, int64_t rows, int64_t width,
                                       float eps, const void* x, int64_t x_stride, const void* w,
                                       const void* bias, void* y, float* mean, float* rstd,
                                       void* stream);

/* Scratch bytes of muon_layer_norm_backward with dw or db. */
MUON_API muon_status_t muon_layer_norm_workspace(int64_t rows, int64_t width, size_t* bytes);

/* The gradient: with xh = (x - mean) * rstd and g = dy * w,
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + residual,
 *   dw = sum over rows of dy * xh, db = sum over rows of dy.
 * residual (nullable): the gradient that goes past the norm, added to dx.  Those of
 * dx (`dtype`), dw and db (w_dtype) that are not NULL are written; the workspace is
 * not needed for dx alone.  Errors: as muon_layer_norm; also INVALID_ARG where dx, dw
 * and db all are NULL, or the workspace is too small or not 256-byte aligned. */
MUON_API muon_status_t muon_layer_norm_backward(int32_t dtype, int32_t w_dtype, int64_t rows,
                                                int64_t width, const void* dy, int64_t dy_stride,
                                                const void* x, int64_t x_stride, const float* mean,
                                                const float* rstd, const void* w,
                                                const void* residual, int64_t residual_stride,
                                                void* dx, void* dw, void* db, void* workspace,
                                                size_t workspace_bytes, void* stream);

/* Scratch bytes of muon_balance_loss. */
MUON_API muon_status_t muon_balance_loss_workspace(int64_t tokens, int32_t experts, size_t* bytes);

/* The load of a router's experts and the loss that evens it out: with p the softmax
 * of a token's logits over all experts,
 *   counts[e] = assignments of indices to e,   live = tokens with a logit above -inf,
 *   loss = coef * experts * sum_e (counts[e] / sum of counts) * (sum over tokens of p[e] / live),
 * coef for a router that is even.  A logit of -inf masks its expert, and a token of
 * which all are masked (padding) has no probabilities and is not live; every index in
 * [0, experts) is an assignment, any other none (muon_gate gives a padded token -1 only);
 * without assignments or live tokens the loss is 0.  A NaN or +inf logit makes the loss
 * NaN.  logits and indices as muon_gate takes and gives them; loss: fp32 [1];
 * counts: int32 [experts]; live: int32 [1].  Errors: INVALID_ARG (as muon_gate; coef
 * not finite; tokens * top_k > 2^31 - 1; workspace), CUDA. */
MUON_API muon_status_t muon_balance_loss(int32_t dtype, int64_t tokens, int32_t experts, int32_t top_k,
                                         float coef, const void* logits, int64_t logits_stride,
                                         const int32_t* indices, float* loss, int32_t* counts,
                                         int32_t* live, void* workspace, size_t workspace_bytes,
                                         void* stream);

/* Its gradient, the counts held fixed: with f = counts / sum of counts,
 *   dlogits = dloss * coef * experts / live * p * (f - <p, f>) + residual.
 * counts and live as muon_balance_loss gave them; dloss: fp32 [1] on the device;
 * residual (nullable): `dtype` [tokens, experts], the logits' gradient through the gate's
 * weights.  A masked expert gets the residual alone; in a token with a NaN or +inf logit
 * all others come out NaN.  dlogits: `dtype`, contiguous.
 * Errors: as muon_balance_loss. */
MUON_API muon_status_t muon_balance_loss_backward(int32_t dtype, int64_t tokens, int32_t experts,
                                                  float coef, const float* dloss, const void* logits,
                                                  int64_t logits_stride, const int32_t* counts,
                                                  const int32_t* live, const void* residual,
                                                  int64_t residual_stride, void* dlogits,
                                                  void* stream);

/* Microscaled 4-bit weights.  A matrix [in, out] is held by rows of its transpose:
 * values [out][B][16 bytes] and scales [out][B bytes], B = ceil(in / 32) blocks of 32
 * steps along in.  A scale byte s is the factor 2^(s - 127), 255 is NaN; an element is
 * four bits, sign, two of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6; element
 * 2 i of a block is in the low half of its byte i.  experts >= 1: that many matrices,
 * one behind the other; 0: one.  values start on 16 bytes.
 *
 * muon_mx_quantize rounds w (`dtype`, stored as muon_linear takes it): a block's scale
 * is the power of two at or below its largest magnitude, over 4 (2^-127 at least), and
 * w / scale goes to the nearest element, ties to the even mantissa, at most 6 (so that
 * magnitudes above 6 of their scale, up to 8, come out as 6).  A block that holds an
 * infinity or a NaN becomes NaN.  Elements past in are 0.  Errors: INVALID_ARG (NULL
 * pointers, sizes, strides, enums, values not on 16 bytes, stream), UNSUPPORTED (more
 * than 2^31 - 1025 blocks in a launch), CUDA. */
MUON_API muon_status_t muon_mx_quantize(int32_t dtype, int32_t w_layout, int32_t experts, int64_t in,
                                        int64_t out, const void* w, int64_t w_stride,
                                        int64_t w_expert_stride, void* values, void* scales,
                                        void* stream);

/* The numbers that values and scales stand for, rounded to `dtype`: w [experts][out][in],
 * contiguous (layout OUT_IN of muon_linear).  Errors: as muon_mx_quantize. */
MUON_API muon_status_t muon_mx_dequantize(int32_t dtype, int32_t experts, int64_t in, int64_t out,
                                          const void* values, const void* scales, void* w,
                                          void* stream);

/* y = act(x' W + bias) + residual for microscaled weights, x' the rows of x rounded as
 * muon_mx_quantize rounds (blocks along in); experts and offsets as in
 * muon_linear_args.  The products of 4-bit numbers and their scales are exact, sums are
 * fp32.  x, bias, residual and y are of `dtype`.  Forward only. */
typedef struct {
  int32_t dtype;       /* muon_dtype_t                                        */
  int32_t activation;  /* muon_activation_t                                   */
  int32_t experts;     /* 0: one matrix; 1 .. MUON_MAX_EXPERTS                */
  int32_t reserved;    /* 0                                                   */
  int64_t rows, in, out;
  int64_t x_stride;    /* row strides in elements                             */
  int64_t residual_stride;
  const void* x;
  const void* w_values;
  const void* w_scales;
  const void* bias;    /* nullable: [out], or [experts, out]                  */
  const void* residual;
  const int32_t* offsets;
  void* y;             /* contiguous [rows, out]                              */
  void* workspace;     /* the rounded rows, and scales in the order of the MMAs (none for few rows) */
  size_t workspace_bytes;
} muon_mx_linear_args;

/* Scratch bytes muon_mx_linear needs for these sizes (pointers are not read).  Errors:
 * INVALID_ARG and UNSUPPORTED as the call itself. */
MUON_API muon_status_t muon_mx_linear_workspace(const muon_mx_linear_args* args, size_t* bytes);

/* Errors, before any launch: INVALID_ARG (NULL args, weights, x or y with rows > 0,
 * offsets NULL with experts > 0; a size, enum or stride out of range; w_values not on
 * 16 bytes; workspace too small or not 256-byte aligned; a stream of another device),
 * UNSUPPORTED (a launch of more than 2^31 - 1025 tiles or blocks), CUDA. */
MUON_API muon_status_t muon_mx_linear(const muon_mx_linear_args* args, void* stream);

/* Synchronises the current device and reads the operators' error word:
 * MUON_OK, or MUON_ERR_TIMEOUT if a kernel of an earlier call gave up a bounded
 * wait (the word is then cleared). */
MUON_API muon_status_t muon_ops_check_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MUON_GB300_OPS_H */
