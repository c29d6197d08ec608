"""The layer operators next to the Muon update: a layer's product with its
epilogue, the same over an expert tensor, the gate, and tokens into expert
order and back, each with its gradient.

Like the plan's steps, these calls work on plain device tensors: no autograd
graph is built, forward and backward are separate calls, and the gradients they
return are what ``MuonPlan.step`` takes.  All arithmetic is in the library's
CUDA kernels (include/muon_ops.h holds the contract of each); this module checks
tensors, allocates outputs and scratch, and marshals pointers.

Every call takes ``stream`` (a ``torch.cuda.Stream`` or a handle; default: the
current stream).  Outputs and scratch belong to that stream in PyTorch's
allocator; a caller who made the inputs on another stream orders the two.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _capi as _c

__all__ = ["linear", "linear_backward", "expert_linear", "expert_linear_backward", "gate", "gate_backward",
           "dispatch", "dispatch_backward", "combine", "combine_backward", "check_ops_error", "ACTIVATIONS"]

ACTIVATIONS = {"none": _c.MUON_ACT_NONE, "relu": _c.MUON_ACT_RELU, "silu": _c.MUON_ACT_SILU,
               "gelu": _c.MUON_ACT_GELU, "gelu_tanh": _c.MUON_ACT_GELU_TANH}
_DTYPES = {torch.float32: _c.MUON_DTYPE_F32, torch.float16: _c.MUON_DTYPE_F16,
           torch.bfloat16: _c.MUON_DTYPE_BF16}


def _dtype(t, what):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} has dtype {t.dtype}, expected float32, float16 or bfloat16")
    return code


def _check(t, what, like, shape, dtype=None):
    if t.shape != torch.Size(shape):
        raise ValueError(f"{what} has shape {list(t.shape)}, expected {list(shape)}")
    if t.dtype != (dtype or like.dtype):
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype or like.dtype}")
    if t.device != like.device:
        raise ValueError(f"{what} must live on {like.device}")


def _contiguous(t, what, like, shape, dtype=None):
    _check(t, what, like, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, what):
    """Row stride of a 2-D tensor whose rows are contiguous and apart."""
    n, width = t.shape
    s0, s1 = t.stride()
    if width > 1 and s1 != 1:
        raise ValueError(f"{what} must have contiguous rows, got strides {list(t.stride())}")
    if n <= 1:
        return width
    if s0 < width:
        raise ValueError(f"{what} has overlapping rows, strides {list(t.stride())}")
    return s0


def _weight(w, what):
    """(layout, row stride as stored) of the last two dims of w."""
    n_in, n_out = w.shape[-2:]
    s0, s1 = w.stride()[-2:]
    if (s1 == 1 or n_out == 1) and (s0 >= n_out or n_in == 1):
        return _c.MUON_W_IN_OUT, s0 if n_in > 1 else n_out
    if (s0 == 1 or n_in == 1) and (s1 >= n_in or n_out == 1):
        return _c.MUON_W_OUT_IN, s1 if n_out > 1 else n_in
    raise ValueError(f"{what} must be contiguous along in or out, got strides {list(w.stride())}")


def _need_cuda(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} must live on a CUDA device")


class _On:
    """The stream and device of one call: its handle, and a context in which
    they are current where they are not already."""

    def __init__(self, like, stream, tensors):
        dev = like.device
        self.other = None
        if stream is None:
            self.handle = torch.cuda.current_stream(dev).cuda_stream
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), dev)
            if s.device != dev:
                raise ValueError(f"stream is on {s.device}, the tensors are on {dev}")
            self.handle = s.cuda_stream
            if s != torch.cuda.current_stream(dev):
                self.other = torch.cuda.stream(s)
                for t in tensors:  # their memory is not handed out again before this call is done with it
                    if t is not None:
                        t.record_stream(s)
        if self.other is None and torch.cuda.current_device() != dev.index:
            self.other = torch.cuda.device(dev)

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()
        return C.c_void_p(self.handle)

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---- linear ----


def _linear_args(x, w, activation, offsets):
    """The arguments both directions share, checked."""
    _need_cuda(x, "x")
    a = _c.muon_linear_args()
    a.dtype = _dtype(x, "x")
    try:
        a.activation = ACTIVATIONS[activation]
    except KeyError:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}") from None
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, in], got {list(x.shape)}")
    lead = 0 if offsets is None else 1
    if w.dim() != 2 + lead or w.shape[-2] != x.shape[1]:
        raise ValueError(f"w must be [{'experts, ' if lead else ''}in, out] with in = {x.shape[1]}, got {list(w.shape)}")
    if w.dtype != x.dtype:
        raise ValueError(f"w has dtype {w.dtype}, expected {x.dtype}")
    if w.device != x.device:
        raise ValueError(f"w must live on {x.device}")
    a.rows, a.out = x.shape[0], w.shape[-1]
    setattr(a, "in", x.shape[1])
    a.x, a.x_stride = x.data_ptr(), _rows(x, "x")
    a.w = w.data_ptr()
    a.w_layout, a.w_stride = _weight(w, "w")
    if lead:
        a.experts = w.shape[0]
        a.w_expert_stride = w.stride(0) if w.shape[0] > 1 else 0
        a.offsets = _contiguous(offsets, "offsets", x, (w.shape[0] + 1,), torch.int32)
    return a


def _scratch(L, a, backward, like):
    n = C.c_size_t()
    _c.check(L.muon_linear_workspace(C.byref(a), backward, C.byref(n)), "muon_linear_workspace")
    if n.value == 0:
        return None
    ws = torch.empty(n.value, dtype=torch.uint8, device=like.device)
    a.workspace, a.workspace_bytes = ws.data_ptr(), n.value
    return ws


def _forward(x, w, offsets, bias, activation, residual, keep_preact, stream):
    a = _linear_args(x, w, activation, offsets)
    rows, out = x.shape[0], w.shape[-1]
    if bias is not None:
        a.bias = _contiguous(bias, "bias", x, (*w.shape[:-2], out))
    if residual is not None:
        _check(residual, "residual", x, (rows, out))
        a.residual, a.residual_stride = residual.data_ptr(), _rows(residual, "residual")
    L = _c.load()
    with _On(x, stream, (x, w, offsets, bias, residual)) as st:
        y = torch.empty((rows, out), dtype=x.dtype, device=x.device)
        a.y = y.data_ptr()
        z = None
        if keep_preact:
            z = torch.empty_like(y)
            a.preact_out = z.data_ptr()
        ws = _scratch(L, a, 0, x)  # noqa: F841  (held until the launch)
        _c.check(L.muon_linear(C.byref(a), st), "muon_linear")
    return (y, z) if keep_preact else y


def _backward(dy, x, w, offsets, preact, activation, dx, dw, bias, stream):
    a = _linear_args(x, w, activation, offsets)
    rows, out = x.shape[0], w.shape[-1]
    _check(dy, "dy", x, (rows, out))
    a.dy, a.dy_stride = dy.data_ptr(), _rows(dy, "dy")
    if a.activation != _c.MUON_ACT_NONE:
        if preact is None:
            raise ValueError(f"preact is needed for activation {activation!r}")
        a.preact = _contiguous(preact, "preact", x, (rows, out))
    if not (dx or dw or bias):
        raise ValueError("nothing to compute: dx, dw and bias are all False")
    L = _c.load()
    gx = gw = gb = None
    with _On(x, stream, (dy, x, w, offsets, preact)) as st:
        if dx:
            gx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            a.dx = gx.data_ptr()
        if dw:  # in w's memory order
            if a.w_layout == _c.MUON_W_IN_OUT:
                gw = torch.empty(w.shape, dtype=w.dtype, device=w.device)
            else:
                gw = torch.empty((*w.shape[:-2], out, w.shape[-2]), dtype=w.dtype, device=w.device).transpose(-1, -2)
            a.dw = gw.data_ptr()
        if bias:
            gb = torch.empty((*w.shape[:-2], out), dtype=x.dtype, device=x.device)
            a.db = gb.data_ptr()
        ws = _scratch(L, a, 1, x)  # noqa: F841  (held until the launch)
        _c.check(L.muon_linear_backward(C.byref(a), st), "muon_linear_backward")
    return gx, gw, gb


def linear(x, w, bias=None, activation="none", residual=None, keep_preact=False, stream=None):
    """y = act(x @ w + bias) + residual for x [rows, in] and w [in, out]; with
    keep_preact (y, z), z = x @ w + bias for the way back.

    w may be stored [out, in] and passed as its transposed view; x and residual
    may have any row stride.  float32, float16 or bfloat16, all tensors of one
    type (16-bit types sum in fp32, fp32 stays fp32)."""
    return _forward(x, w, None, bias, activation, residual, keep_preact, stream)


def linear_backward(dy, x, w, preact=None, activation="none", dx=True, dw=True, bias=False, stream=None):
    """(dx, dw, db) of linear for the gradient dy of its result; those not asked
    for are None.  dw has w's shape and memory order.  The residual's gradient
    is dy itself."""
    return _backward(dy, x, w, None, preact, activation, dx, dw, bias, stream)


def expert_linear(x, offsets, w, bias=None, activation="none", residual=None, keep_preact=False, stream=None):
    """linear over an expert tensor w [experts, in, out]: rows
    offsets[e] .. offsets[e + 1] - 1 of x (int32, on the device, as ``dispatch``
    gives them) go through w[e] and bias[e].  Rows from offsets[-1] on come out
    zero."""
    return _forward(x, w, _given(offsets), bias, activation, residual, keep_preact, stream)


def expert_linear_backward(dy, x, offsets, w, preact=None, activation="none", dx=True, dw=True, bias=False,
                           stream=None):
    """(dx, dw, db) of expert_linear; an expert without rows gets zero dw and db."""
    return _backward(dy, x, w, _given(offsets), preact, activation, dx, dw, bias, stream)


def _given(offsets):
    if offsets is None:
        raise ValueError("offsets is needed")
    return offsets


# ---- gate ----


def _gate_check(logits, top_k):
    _need_cuda(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [tokens, experts], got {list(logits.shape)}")
    return _dtype(logits, "logits"), _rows(logits, "logits")


def gate(logits, top_k, renormalize=True, stream=None):
    """(indices int32, weights float32), [tokens, top_k] each: the experts with
    the largest logits in falling order (ties: the lower index) and their
    softmax weights, over the chosen experts (renormalize) or over all.  A
    logit of -inf masks an expert; places that no open expert is left for get
    index -1 and weight 0."""
    code, stride = _gate_check(logits, top_k)
    tokens, experts = logits.shape
    L = _c.load()
    with _On(logits, stream, (logits,)) as st:
        idx = torch.empty((tokens, int(top_k)), dtype=torch.int32, device=logits.device)
        wts = torch.empty((tokens, int(top_k)), dtype=torch.float32, device=logits.device)
        _c.check(L.muon_gate(code, tokens, experts, int(top_k), int(renormalize), logits.data_ptr(), stride,
                             idx.data_ptr(), wts.data_ptr(), st), "muon_gate")
    return idx, wts


def gate_backward(dweights, logits, indices, renormalize=True, stream=None):
    """The gradient of gate's logits for that of its weights, the choice held
    fixed (indices as gate gave them)."""
    if indices.dim() != 2:
        raise ValueError(f"indices must be [tokens, top_k], got {list(indices.shape)}")
    top_k = indices.shape[1]
    code, stride = _gate_check(logits, top_k)
    tokens, experts = logits.shape
    ip = _contiguous(indices, "indices", logits, (tokens, top_k), torch.int32)
    dp = _contiguous(dweights, "dweights", logits, (tokens, top_k), torch.float32)
    L = _c.load()
    with _On(logits, stream, (dweights, logits, indices)) as st:
        out = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
        _c.check(L.muon_gate_backward(code, tokens, experts, top_k, int(renormalize), dp, logits.data_ptr(),
                                      stride, ip, out.data_ptr(), st), "muon_gate_backward")
    return out


# ---- tokens into expert order and back ----


def _matrix(t, what):
    _need_cuda(t, what)
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D, got {list(t.shape)}")
    return _dtype(t, what), _rows(t, what)


def _slots(slot, like):
    if slot.dim() != 2:
        raise ValueError(f"slot must be [tokens, top_k], got {list(slot.shape)}")
    return _contiguous(slot, "slot", like, slot.shape, torch.int32)


def dispatch(x, indices, n_experts, stream=None):
    """(xs, slot, offsets): the rows of x [tokens, hidden] in expert order.

    Assignment (t, j) of indices [tokens, top_k] (int32 or int64) goes to row
    slot[t, j] of xs [tokens * top_k, hidden]: by expert, then t, then j.  An
    index outside [0, n_experts) drops its assignment (slot -1).  Expert e owns
    rows offsets[e] .. offsets[e + 1] - 1; rows that no expert owns are zero."""
    code, stride = _matrix(x, "x")
    tokens, hidden = x.shape
    if indices.dim() != 2 or indices.shape[0] != tokens:
        raise ValueError(f"indices must be [tokens, top_k] with tokens = {tokens}, got {list(indices.shape)}")
    if indices.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"indices has dtype {indices.dtype}, expected int32 or int64")
    top_k = indices.shape[1]
    ip = _contiguous(indices, "indices", x, indices.shape, indices.dtype)
    L = _c.load()
    n = C.c_size_t()
    _c.check(L.muon_dispatch_workspace(tokens, top_k, int(n_experts), C.byref(n)), "muon_dispatch_workspace")
    dev = x.device
    with _On(x, stream, (x, indices)) as st:
        xs = torch.empty((tokens * top_k, hidden), dtype=x.dtype, device=dev)
        slot = torch.empty((tokens, top_k), dtype=torch.int32, device=dev)
        offsets = torch.empty(int(n_experts) + 1, dtype=torch.int32, device=dev)
        ws = torch.empty(n.value, dtype=torch.uint8, device=dev) if n.value else None
        _c.check(L.muon_dispatch(code, tokens, hidden, top_k, int(n_experts), x.data_ptr(), stride, ip,
                                 8 * indices.element_size(), xs.data_ptr(), slot.data_ptr(), offsets.data_ptr(),
                                 _ptr(ws), n.value, st), "muon_dispatch")
    return xs, slot, offsets


def dispatch_backward(dxs, slot, stream=None):
    """dx[t] = sum over j of dxs[slot[t, j]]."""
    code, stride = _matrix(dxs, "dxs")
    sp = _slots(slot, dxs)
    tokens, top_k = slot.shape
    if dxs.shape[0] != tokens * top_k:
        raise ValueError(f"dxs must have tokens * top_k = {tokens * top_k} rows, got {dxs.shape[0]}")
    L = _c.load()
    with _On(dxs, stream, (dxs, slot)) as st:
        dx = torch.empty((tokens, dxs.shape[1]), dtype=dxs.dtype, device=dxs.device)
        _c.check(L.muon_dispatch_backward(code, tokens, dxs.shape[1], top_k, dxs.data_ptr(), stride, sp,
                                          dx.data_ptr(), st), "muon_dispatch_backward")
    return dx


def combine(ys, slot, weights, residual=None, stream=None):
    """y[t] = sum over j of weights[t, j] * ys[slot[t, j]], + residual[t]."""
    code, stride = _matrix(ys, "ys")
    sp = _slots(slot, ys)
    tokens, top_k = slot.shape
    if ys.shape[0] != tokens * top_k:
        raise ValueError(f"ys must have tokens * top_k = {tokens * top_k} rows, got {ys.shape[0]}")
    wp = _contiguous(weights, "weights", ys, slot.shape, torch.float32)
    hidden, r_stride = ys.shape[1], 0
    if residual is not None:
        _check(residual, "residual", ys, (tokens, hidden))
        r_stride = _rows(residual, "residual")
    L = _c.load()
    with _On(ys, stream, (ys, slot, weights, residual)) as st:
        y = torch.empty((tokens, hidden), dtype=ys.dtype, device=ys.device)
        _c.check(L.muon_combine(code, tokens, hidden, top_k, ys.data_ptr(), stride, sp, wp, _ptr(residual),
                                r_stride, y.data_ptr(), st), "muon_combine")
    return y


def combine_backward(dy, ys, slot, offsets, weights, stream=None):
    """(dys, dweights): dys[slot[t, j]] = weights[t, j] * dy[t], zero in the rows
    that no expert owns, and dweights[t, j] = <ys[slot[t, j]], dy[t]> in fp32
    (offsets as ``dispatch`` gave them)."""
    code, stride = _matrix(ys, "ys")
    sp = _slots(slot, ys)
    tokens, top_k = slot.shape
    if ys.shape[0] != tokens * top_k:
        raise ValueError(f"ys must have tokens * top_k = {tokens * top_k} rows, got {ys.shape[0]}")
    _check(dy, "dy", ys, (tokens, ys.shape[1]))
    d_stride = _rows(dy, "dy")
    wp = _contiguous(weights, "weights", ys, slot.shape, torch.float32)
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets must be [experts + 1], got {list(offsets.shape)}")
    op = _contiguous(offsets, "offsets", ys, offsets.shape, torch.int32)
    L = _c.load()
    with _On(ys, stream, (dy, ys, slot, offsets, weights)) as st:
        dys = torch.empty(ys.shape, dtype=ys.dtype, device=ys.device)
        dwts = torch.empty(slot.shape, dtype=torch.float32, device=ys.device)
        _c.check(L.muon_combine_backward(code, tokens, ys.shape[1], top_k, offsets.shape[0] - 1, dy.data_ptr(),
                                         d_stride, ys.data_ptr(), stride, sp, op, wp, dys.data_ptr(),
                                         dwts.data_ptr(), st), "muon_combine_backward")
    return dys, dwts


def check_ops_error() -> None:
    """Synchronises the current device; raises MuonError if a kernel of an
    earlier call gave up a bounded wait."""
    _c.check(_c.load().muon_ops_check_error(), "muon_ops_check_error")
