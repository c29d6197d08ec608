"""The layer operators next to the Muon update: a layer's product with its
epilogue, the same over an expert tensor, the gate, tokens into expert order and
back, the layer norm and a router's balance loss, each with its gradient; and for
serving, weights in microscaled 4-bit numbers and the products that read them.

Like the plan's steps, these calls work on plain device tensors: no autograd
graph is built, forward and backward are separate calls, and the gradients they
return are what ``MuonPlan.step`` takes.  Where autograd is recording, a tensor
that requires grad is refused (a ``torch.autograd.Function`` may call them).  All arithmetic is in the library's
CUDA kernels (include/muon_ops.h holds the contract of each); this module checks
tensors, allocates outputs and scratch, and marshals pointers.

Every call takes ``stream=`` (a ``torch.cuda.Stream`` or a handle; default: the
current stream).  Outputs and scratch belong to that stream in PyTorch's
allocator; a caller who made the inputs on another stream orders the two.  The
tensors live on the current device.
"""
from __future__ import annotations

import ctypes as C
import functools
import struct

import torch

from . import _capi as _c

__all__ = ["linear", "linear_backward", "expert_linear", "expert_linear_backward", "gate", "gate_backward",
           "dispatch", "dispatch_backward", "combine", "combine_backward", "layer_norm", "layer_norm_backward",
           "balance_loss", "balance_loss_backward", "mx_quantize", "mx_dequantize", "mx_linear", "mx_expert_linear",
           "check_ops_error", "ACTIVATIONS"]

ACTIVATIONS = {"none": _c.MUON_ACT_NONE, "relu": _c.MUON_ACT_RELU, "silu": _c.MUON_ACT_SILU,
               "gelu": _c.MUON_ACT_GELU, "gelu_tanh": _c.MUON_ACT_GELU_TANH}
_DTYPES = {torch.float32: _c.MUON_DTYPE_F32, torch.float16: _c.MUON_DTYPE_F16,
           torch.bfloat16: _c.MUON_DTYPE_BF16}
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_empty = torch.empty

# A call on small tensors is bound by this module's own time, so the checks
# read each property once, the argument structure is packed in one step
# (muon_linear_args: 4 int32, 8 int64, 13 pointers, a size), and scratch sizes
# are remembered per problem.
_PACK = struct.Struct("=4i8q14Q").pack
assert struct.calcsize("=4i8q14Q") == C.sizeof(_c.muon_linear_args)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
_grad_enabled = torch.is_grad_enabled
_Tensor = torch.Tensor


def _operator(op):
    """Adds ``stream`` to an operator that runs on the current stream, and refuses
    tensors whose gradient autograd would expect and not get."""

    def refuse(args, kw):
        named = (*zip(op.__code__.co_varnames, args), *kw.items())
        name = next(n for n, t in named if isinstance(t, _Tensor) and t.requires_grad)
        raise ValueError(f"{name} requires grad, but {op.__name__} builds no autograd graph: detach it or call under "
                         "torch.no_grad(); gradients come from the _backward calls")

    @functools.wraps(op)
    def call(*args, stream=None, **kw):
        if _grad_enabled():
            for t in args:
                if isinstance(t, _Tensor) and t.requires_grad:
                    refuse(args, kw)
            for t in kw.values():
                if isinstance(t, _Tensor) and t.requires_grad:
                    refuse(args, kw)
        if stream is None:
            return op(*args, **kw)
        like = next((t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if like is None or not like.is_cuda:
            raise ValueError("the tensors must live on a CUDA device")
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), like.device)
        if s.device != like.device:
            raise ValueError(f"stream is on {s.device}, the tensors are on {like.device}")
        if s != torch.cuda.current_stream(like.device):
            for t in (*args, *kw.values()):  # not handed out again before this call is done with it
                if isinstance(t, torch.Tensor):
                    t.record_stream(s)
        with torch.cuda.stream(s):
            return op(*args, **kw)

    return call


def _start(t, what, dims):
    """(device index, current stream, dtype code) of an operator's first tensor."""
    if t.dim() != dims:
        raise ValueError(f"{what} must be {dims}-D, got {list(t.shape)}")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} has dtype {t.dtype}, expected float32, float16 or bfloat16")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must live on a CUDA device")
    if dev != _current_device():
        raise ValueError(f"{what} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev, _raw_stream(dev), code


def _check(t, what, dev, dtype, shape):
    if t.shape != shape:
        raise ValueError(f"{what} has shape {list(t.shape)}, expected {list(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{what} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what} must live on cuda:{dev}")


def _contiguous(t, what, dev, dtype, shape):
    """Address of a contiguous tensor of this type and shape."""
    _check(t, what, dev, dtype, shape)
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


def _weight(w, n_in, n_out):
    """(layout, row stride as stored) of the last two dims of w."""
    *_, s0, s1 = w.stride()
    if (s1 == 1 or n_out == 1) and (s0 >= n_out or n_in == 1):
        return _c.MUON_W_IN_OUT, s0 if n_in > 1 else n_out
    if (s0 == 1 or n_in == 1) and (s1 >= n_in or n_out == 1):
        return _c.MUON_W_OUT_IN, s1 if n_out > 1 else n_in
    raise ValueError(f"w must be contiguous along in or out, got strides {list(w.stride())}")


# ---- linear ----

_scratch_sizes = {}


@functools.lru_cache(maxsize=None)
def _linear_call(backward):
    """muon_linear(_backward) taking the packed structure."""
    return C.CFUNCTYPE(C.c_int, C.c_char_p, C.c_void_p)(
        ("muon_linear_backward" if backward else "muon_linear", _c.load()))


def _run(backward, dev, stream, head, strides, ptrs):
    """One call: head = dtype .. out, then strides, then pointers x .. db."""
    # what the size depends on: the problem, 16-byte alignment, and the gradients asked for
    x, w = ptrs[0], ptrs[1]
    if backward:
        key = (head, strides, x & 15, w & 15, ptrs[6] & 15, ptrs[9] > 0, ptrs[10] > 0, ptrs[11] > 0)
    else:
        key = (head, strides, x & 15, w & 15)
    size = _scratch_sizes.get(key)
    if size is None:
        n = C.c_size_t()
        a = _c.muon_linear_args.from_buffer_copy(_PACK(*head, *strides, *ptrs, 0, 0))
        _c.check(_c.load().muon_linear_workspace(C.byref(a), int(backward), C.byref(n)), "muon_linear_workspace")
        if len(_scratch_sizes) >= 4096:
            _scratch_sizes.clear()
        size = _scratch_sizes[key] = n.value
    ws = _empty(size, dtype=torch.uint8, device=dev) if size else None
    st = _linear_call(backward)(_PACK(*head, *strides, *ptrs, ws.data_ptr() if size else 0, size), stream)
    if st:
        _c.check(st, "muon_linear_backward" if backward else "muon_linear")


def _problem(x, w, offsets, activation):
    """What both directions share, checked."""
    dev, stream, code = _start(x, "x", 2)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    rows, n_in = x.shape
    shape = w.shape
    lead = 0 if offsets is None else 1
    if len(shape) != 2 + lead or shape[-2] != n_in:
        raise ValueError(f"w must be [{'experts, ' if lead else ''}in, out] with in = {n_in}, got {list(shape)}")
    if w.dtype != x.dtype or w.get_device() != dev:
        raise ValueError(f"w must be {x.dtype} on cuda:{dev}, got {w.dtype} on {w.device}")
    n_out = shape[-1]
    layout, w_stride = _weight(w, n_in, n_out)
    experts = off = e_stride = 0
    if lead:
        experts = shape[0]
        e_stride = w.stride(0) if experts > 1 else 0
        off = _contiguous(offsets, "offsets", dev, _I32, (experts + 1,))
    return dev, stream, (code, act, experts, layout, rows, n_in, n_out), w_stride, e_stride, off


def _forward(x, w, offsets, bias, activation, residual, keep_preact):
    dev, stream, head, w_stride, e_stride, off = _problem(x, w, offsets, activation)
    dtype, rows, out = x.dtype, head[4], head[6]
    bp = rp = r_stride = 0
    if bias is not None:
        bp = _contiguous(bias, "bias", dev, dtype, (out,) if offsets is None else (head[2], out))
    if residual is not None:
        _check(residual, "residual", dev, dtype, (rows, out))
        rp, r_stride = residual.data_ptr(), _rows(residual, "residual")
    y = _empty((rows, out), dtype=dtype, device=dev)
    z = _empty((rows, out), dtype=dtype, device=dev) if keep_preact else None
    _run(False, dev, stream, head, (_rows(x, "x"), w_stride, e_stride, r_stride, 0),
         (x.data_ptr(), w.data_ptr(), bp, rp, off, 0, 0, y.data_ptr(), z.data_ptr() if keep_preact else 0, 0, 0, 0))
    return (y, z) if keep_preact else y


def _backward(dy, x, w, offsets, preact, activation, dx, dw, bias):
    dev, stream, head, w_stride, e_stride, off = _problem(x, w, offsets, activation)
    dtype, experts, rows, n_in, out = x.dtype, head[2], head[4], head[5], head[6]
    _check(dy, "dy", dev, dtype, (rows, out))
    zp = 0
    if head[1] != _c.MUON_ACT_NONE:
        if preact is None:
            raise ValueError(f"preact is needed for activation {activation!r}")
        zp = _contiguous(preact, "preact", dev, dtype, (rows, out))
    if not (dx or dw or bias):
        raise ValueError("nothing to compute: dx, dw and bias are all False")
    lead = () if offsets is None else (experts,)
    gx = gw = gb = None
    xp = wp = bp = 0
    if dx:
        gx = _empty((rows, n_in), dtype=dtype, device=dev)
        xp = gx.data_ptr()
    if dw:  # in w's memory order
        if head[3] == _c.MUON_W_IN_OUT:
            gw = _empty((*lead, n_in, out), dtype=dtype, device=dev)
        else:
            gw = _empty((*lead, out, n_in), dtype=dtype, device=dev).transpose(-1, -2)
        wp = gw.data_ptr()
    if bias:
        gb = _empty((*lead, out), dtype=dtype, device=dev)
        bp = gb.data_ptr()
    _run(True, dev, stream, head, (_rows(x, "x"), w_stride, e_stride, 0, _rows(dy, "dy")),
         (x.data_ptr(), w.data_ptr(), 0, 0, off, zp, dy.data_ptr(), 0, 0, xp, wp, bp))
    return gx, gw, gb


@_operator
def linear(x, w, bias=None, activation="none", residual=None, keep_preact=False):
    """y = act(x @ w + bias) + residual for x [rows, in] and w [in, out]; with
    keep_preact (y, z), z = x @ w + bias for the way back.

    w may be stored [out, in] and passed as its transposed view; x and residual
    may have any row stride.  float32, float16 or bfloat16, all tensors of one
    type (16-bit types sum in fp32, fp32 stays fp32)."""
    return _forward(x, w, None, bias, activation, residual, keep_preact)


@_operator
def linear_backward(dy, x, w, preact=None, activation="none", dx=True, dw=True, bias=False):
    """(dx, dw, db) of linear for the gradient dy of its result; those not asked
    for are None.  dw has w's shape and memory order.  The residual's gradient
    is dy itself."""
    return _backward(dy, x, w, None, preact, activation, dx, dw, bias)


@_operator
def expert_linear(x, offsets, w, bias=None, activation="none", residual=None, keep_preact=False):
    """linear over an expert tensor w [experts, in, out]: rows
    offsets[e] .. offsets[e + 1] - 1 of x (int32, on the device, as ``dispatch``
    gives them) go through w[e] and bias[e].  Rows before offsets[0] and from
    offsets[-1] on come out zero."""
    return _forward(x, w, _given(offsets), bias, activation, residual, keep_preact)


@_operator
def expert_linear_backward(dy, x, offsets, w, preact=None, activation="none", dx=True, dw=True, bias=False):
    """(dx, dw, db) of expert_linear; an expert without rows gets zero dw and db."""
    return _backward(dy, x, w, _given(offsets), preact, activation, dx, dw, bias)


def _given(offsets):
    if offsets is None:
        raise ValueError("offsets is needed")
    return offsets


def _int32(n):
    """n as the C ABI's int32 arguments take it: what does not fit becomes a value
    that is out of every range, not another number."""
    n = int(n)
    return n if -1 <= n <= 0x7fffffff else -1


# ---- gate ----


@_operator
def gate(logits, top_k, renormalize=True):
    """(indices int32, weights float32), [tokens, top_k] each: the experts with
    the largest logits in falling order (ties: the lower index) and their
    softmax weights, over the chosen experts (renormalize) or over all.  A
    logit of -inf masks an expert; places that no open expert is left for get
    index -1 and weight 0."""
    dev, stream, code = _start(logits, "logits", 2)
    tokens, experts = logits.shape
    top_k = _int32(top_k)
    k = top_k if 0 < top_k <= experts else 0  # refused below, with nothing allocated for it
    idx = _empty((tokens, k), dtype=_I32, device=dev)
    wts = _empty((tokens, k), dtype=_F32, device=dev)
    st = _c.load().muon_gate(code, tokens, _int32(experts), top_k, renormalize, logits.data_ptr(),
                             _rows(logits, "logits"), idx.data_ptr(), wts.data_ptr(), stream)
    if st:
        _c.check(st, "muon_gate")
    return idx, wts


@_operator
def gate_backward(dweights, logits, indices, renormalize=True):
    """The gradient of gate's logits for that of its weights, the choice held
    fixed (indices as gate gave them)."""
    dev, stream, code = _start(logits, "logits", 2)
    tokens, experts = logits.shape
    if indices.dim() != 2:
        raise ValueError(f"indices must be [tokens, top_k], got {list(indices.shape)}")
    top_k = indices.shape[1]
    ip = _contiguous(indices, "indices", dev, _I32, (tokens, top_k))
    dp = _contiguous(dweights, "dweights", dev, _F32, (tokens, top_k))
    out = _empty((tokens, experts), dtype=logits.dtype, device=dev)
    st = _c.load().muon_gate_backward(code, tokens, _int32(experts), top_k, renormalize, dp, logits.data_ptr(),
                                      _rows(logits, "logits"), ip, out.data_ptr(), stream)
    if st:
        _c.check(st, "muon_gate_backward")
    return out


# ---- tokens into expert order and back ----


def _slots(slot, rows, what, dev):
    """(address, tokens, top_k) of the slots of `rows` rows in expert order."""
    if slot.dim() != 2:
        raise ValueError(f"slot must be [tokens, top_k], got {list(slot.shape)}")
    tokens, top_k = slot.shape
    if rows != tokens * top_k:
        raise ValueError(f"{what} must have tokens * top_k = {tokens * top_k} rows, got {rows}")
    return _contiguous(slot, "slot", dev, _I32, (tokens, top_k)), tokens, top_k


@_operator
def dispatch(x, indices, n_experts):
    """(xs, slot, offsets): the rows of x [tokens, hidden] in expert order.

    Assignment (t, j) of indices [tokens, top_k] (int32 or int64) goes to row
    slot[t, j] of xs [tokens * top_k, hidden]: by expert, then t, then j.  An
    index outside [0, n_experts) drops its assignment (slot -1).  Expert e owns
    rows offsets[e] .. offsets[e + 1] - 1; rows that no expert owns are zero."""
    dev, stream, code = _start(x, "x", 2)
    tokens, hidden = x.shape
    if indices.dim() != 2 or indices.shape[0] != tokens:
        raise ValueError(f"indices must be [tokens, top_k] with tokens = {tokens}, got {list(indices.shape)}")
    if indices.dtype != _I32 and indices.dtype != _I64:
        raise ValueError(f"indices has dtype {indices.dtype}, expected int32 or int64")
    top_k, n_experts = indices.shape[1], _int32(n_experts)
    ip = _contiguous(indices, "indices", dev, indices.dtype, indices.shape)
    L = _c.load()
    n = C.c_size_t()
    st = L.muon_dispatch_workspace(tokens, top_k, n_experts, C.byref(n))
    if st:
        _c.check(st, "muon_dispatch_workspace")
    size = n.value
    xs = _empty((tokens * top_k, hidden), dtype=x.dtype, device=dev)
    slot = _empty((tokens, top_k), dtype=_I32, device=dev)
    offsets = _empty(n_experts + 1, dtype=_I32, device=dev)
    ws = _empty(size, dtype=torch.uint8, device=dev) if size else None
    st = L.muon_dispatch(code, tokens, hidden, top_k, n_experts, x.data_ptr(), _rows(x, "x"), ip,
                         32 if indices.dtype == _I32 else 64, xs.data_ptr(), slot.data_ptr(), offsets.data_ptr(),
                         ws.data_ptr() if size else None, size, stream)
    if st:
        _c.check(st, "muon_dispatch")
    return xs, slot, offsets


@_operator
def dispatch_backward(dxs, slot):
    """dx[t] = sum over j of dxs[slot[t, j]]."""
    dev, stream, code = _start(dxs, "dxs", 2)
    rows, hidden = dxs.shape
    sp, tokens, top_k = _slots(slot, rows, "dxs", dev)
    dx = _empty((tokens, hidden), dtype=dxs.dtype, device=dev)
    st = _c.load().muon_dispatch_backward(code, tokens, hidden, top_k, dxs.data_ptr(), _rows(dxs, "dxs"), sp,
                                          dx.data_ptr(), stream)
    if st:
        _c.check(st, "muon_dispatch_backward")
    return dx


@_operator
def combine(ys, slot, weights, residual=None):
    """y[t] = sum over j of weights[t, j] * ys[slot[t, j]], + residual[t]."""
    dev, stream, code = _start(ys, "ys", 2)
    rows, hidden = ys.shape
    sp, tokens, top_k = _slots(slot, rows, "ys", dev)
    wp = _contiguous(weights, "weights", dev, _F32, (tokens, top_k))
    rp, r_stride = None, 0
    if residual is not None:
        _check(residual, "residual", dev, ys.dtype, (tokens, hidden))
        rp, r_stride = residual.data_ptr(), _rows(residual, "residual")
    y = _empty((tokens, hidden), dtype=ys.dtype, device=dev)
    st = _c.load().muon_combine(code, tokens, hidden, top_k, ys.data_ptr(), _rows(ys, "ys"), sp, wp, rp, r_stride,
                                y.data_ptr(), stream)
    if st:
        _c.check(st, "muon_combine")
    return y


@_operator
def combine_backward(dy, ys, slot, offsets, weights):
    """(dys, dweights): dys[slot[t, j]] = weights[t, j] * dy[t], zero in the rows
    that no expert owns, and dweights[t, j] = <ys[slot[t, j]], dy[t]> in fp32
    (offsets as ``dispatch`` gave them)."""
    dev, stream, code = _start(ys, "ys", 2)
    rows, hidden = ys.shape
    sp, tokens, top_k = _slots(slot, rows, "ys", dev)
    _check(dy, "dy", dev, ys.dtype, (tokens, hidden))
    wp = _contiguous(weights, "weights", dev, _F32, (tokens, top_k))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets must be [experts + 1], got {list(offsets.shape)}")
    op = _contiguous(offsets, "offsets", dev, _I32, offsets.shape)
    dys = _empty((rows, hidden), dtype=ys.dtype, device=dev)
    dwts = _empty((tokens, top_k), dtype=_F32, device=dev)
    st = _c.load().muon_combine_backward(code, tokens, hidden, top_k, _int32(offsets.shape[0] - 1), dy.data_ptr(),
                                         _rows(dy, "dy"), ys.data_ptr(), _rows(ys, "ys"), sp, op, wp,
                                         dys.data_ptr(), dwts.data_ptr(), stream)
    if st:
        _c.check(st, "muon_combine_backward")
    return dys, dwts


# ---- layer norm ----


@functools.lru_cache(maxsize=4096)
def _scratch_size(call, *problem):
    """Scratch bytes that the library's `call` gives for these sizes."""
    n = C.c_size_t()
    _c.check(getattr(_c.load(), call)(*problem, C.byref(n)), call)
    return n.value


def _norm_weight(w, what, dev, dtype, width, like=None):
    """(address, dtype code) of a norm's weight, of x's type or float32."""
    if w.dtype != dtype and w.dtype != _F32:
        raise ValueError(f"{what} has dtype {w.dtype}, expected {dtype} or {_F32}")
    return _contiguous(w, what, dev, w.dtype if like is None else like, (width,)), _DTYPES[w.dtype]


@_operator
def layer_norm(x, w=None, bias=None, eps=1e-5, keep_stats=False):
    """y[t] = (x[t] - mean) / sqrt(var + eps) * w + bias over each row of x [rows,
    width]; with keep_stats (y, mean, rstd), float32 [rows] each, for the way
    back.

    w and bias [width] are of x's type or float32, both alike; x may have any row
    stride."""
    dev, stream, code = _start(x, "x", 2)
    rows, width = x.shape
    wp = bp = None
    w_code = code
    if w is not None:
        wp, w_code = _norm_weight(w, "w", dev, x.dtype, width)
    if bias is not None:
        bp, w_code = _norm_weight(bias, "bias", dev, x.dtype, width, None if w is None else w.dtype)
    y = _empty((rows, width), dtype=x.dtype, device=dev)
    mean = rstd = mp = sp = None
    if keep_stats:
        mean, rstd = _empty(rows, dtype=_F32, device=dev), _empty(rows, dtype=_F32, device=dev)
        mp, sp = mean.data_ptr(), rstd.data_ptr()
    st = _c.load().muon_layer_norm(code, w_code, rows, width, eps, x.data_ptr(), _rows(x, "x"), wp, bp, y.data_ptr(),
                                   mp, sp, stream)
    if st:
        _c.check(st, "muon_layer_norm")
    return (y, mean, rstd) if keep_stats else y


@_operator
def layer_norm_backward(dy, x, mean, rstd, w=None, residual=None, dx=True, dw=True, bias=False):
    """(dx, dw, db) of layer_norm for the gradient dy of its result, with the
    statistics that keep_stats gave; those not asked for are None.  residual, the
    gradient that goes past the norm, is added to dx.  dw and db are of w's type
    (x's without w)."""
    dev, stream, code = _start(x, "x", 2)
    rows, width = x.shape
    dtype = x.dtype
    _check(dy, "dy", dev, dtype, (rows, width))
    mp, sp = _contiguous(mean, "mean", dev, _F32, (rows,)), _contiguous(rstd, "rstd", dev, _F32, (rows,))
    wp, w_code, w_dtype = None, code, dtype
    if w is not None:
        wp, w_code = _norm_weight(w, "w", dev, dtype, width)
        w_dtype = w.dtype
    if not (dx or dw or bias):
        raise ValueError("nothing to compute: dx, dw and bias are all False")
    rp, r_stride = None, 0
    if residual is not None:
        if not dx:
            raise ValueError("residual is added to dx, which is not asked for")
        _check(residual, "residual", dev, dtype, (rows, width))
        rp, r_stride = residual.data_ptr(), _rows(residual, "residual")
    gx = _empty((rows, width), dtype=dtype, device=dev) if dx else None
    gw = _empty(width, dtype=w_dtype, device=dev) if dw else None
    gb = _empty(width, dtype=w_dtype, device=dev) if bias else None
    size = _scratch_size("muon_layer_norm_workspace", rows, width) if dw or bias else 0
    ws = _empty(size, dtype=torch.uint8, device=dev) if size else None
    st = _c.load().muon_layer_norm_backward(
        code, w_code, rows, width, dy.data_ptr(), _rows(dy, "dy"), x.data_ptr(), _rows(x, "x"), mp, sp, wp, rp, r_stride,
        gx.data_ptr() if dx else None, gw.data_ptr() if dw else None, gb.data_ptr() if bias else None,
        ws.data_ptr() if size else None, size, stream)
    if st:
        _c.check(st, "muon_layer_norm_backward")
    return gx, gw, gb


# ---- balance loss ----


@_operator
def balance_loss(logits, indices, coef=1.0):
    """(loss, counts, live): coef * experts * sum over experts of the share of the
    assignments that an expert got and its mean probability (softmax over all
    experts), coef itself for an even router; the assignments of each expert
    (int32 [experts]) and the tokens counted (int32 []).

    logits [tokens, experts] and indices [tokens, top_k] as ``gate`` takes and gives
    them.  A logit of -inf masks its expert; a token with none left (padding) is not
    counted; an index in [0, experts) is an assignment, any other none."""
    dev, stream, code = _start(logits, "logits", 2)
    tokens, experts = logits.shape
    if indices.dim() != 2:
        raise ValueError(f"indices must be [tokens, top_k], got {list(indices.shape)}")
    top_k = indices.shape[1]
    ip = _contiguous(indices, "indices", dev, _I32, (tokens, top_k))
    size = _scratch_size("muon_balance_loss_workspace", tokens, _int32(experts))
    ws = _empty(size, dtype=torch.uint8, device=dev) if size else None
    loss, live = _empty((), dtype=_F32, device=dev), _empty((), dtype=_I32, device=dev)
    counts = _empty(experts, dtype=_I32, device=dev)
    st = _c.load().muon_balance_loss(code, tokens, experts, _int32(top_k), coef, logits.data_ptr(),
                                     _rows(logits, "logits"), ip, loss.data_ptr(), counts.data_ptr(), live.data_ptr(),
                                     ws.data_ptr() if size else None, size, stream)
    if st:
        _c.check(st, "muon_balance_loss")
    return loss, counts, live


@_operator
def balance_loss_backward(dloss, logits, counts, live, coef=1.0, residual=None):
    """The gradient of balance_loss's logits for that of its loss (float32, one
    element on the device), the counts held fixed, plus residual (``gate_backward``'s
    gradient of the same logits)."""
    dev, stream, code = _start(logits, "logits", 2)
    tokens, experts = logits.shape
    dp = _one(dloss, "dloss", dev, _F32)
    np_ = _one(live, "live", dev, _I32)
    cp = _contiguous(counts, "counts", dev, _I32, (experts,))
    rp, r_stride = None, 0
    if residual is not None:
        _check(residual, "residual", dev, logits.dtype, (tokens, experts))
        rp, r_stride = residual.data_ptr(), _rows(residual, "residual")
    out = _empty((tokens, experts), dtype=logits.dtype, device=dev)
    st = _c.load().muon_balance_loss_backward(code, tokens, _int32(experts), coef, dp, logits.data_ptr(),
                                              _rows(logits, "logits"), cp, np_, rp, r_stride, out.data_ptr(), stream)
    if st:
        _c.check(st, "muon_balance_loss_backward")
    return out


def _one(t, what, dev, dtype):
    """Address of a tensor of one element."""
    if t.numel() != 1:
        raise ValueError(f"{what} must have one element, got {list(t.shape)}")
    _check(t, what, dev, dtype, t.shape)
    return t.data_ptr()


# ---- microscaled 4-bit weights ----

_U8 = torch.uint8
_MX_PACK = struct.Struct("=4i5q9Q").pack
assert struct.calcsize("=4i5q9Q") == C.sizeof(_c.muon_mx_linear_args)


@functools.lru_cache(maxsize=None)
def _mx_call():
    """muon_mx_linear taking the packed structure."""
    return C.CFUNCTYPE(C.c_int, C.c_char_p, C.c_void_p)(("muon_mx_linear", _c.load()))


@functools.lru_cache(maxsize=4096)
def _mx_scratch_size(code, experts, rows, n_in, out):
    n = C.c_size_t()
    a = _c.muon_mx_linear_args.from_buffer_copy(
        _MX_PACK(code, 0, _int32(experts), 0, rows, n_in, out, n_in, 0, *(0,) * 9))
    _c.check(_c.load().muon_mx_linear_workspace(C.byref(a), C.byref(n)), "muon_mx_linear_workspace")
    return n.value


@_operator
def mx_quantize(w):
    """(values, scales), uint8: w [in, out] or [experts, in, out] in microscaled 4-bit
    numbers, in blocks of 32 along in.

    values is [.., out, 16 * blocks], two numbers to a byte, scales [.., out, blocks],
    with blocks = ceil(in / 32): the power of two 2^(scale - 127) at or below a block's
    largest magnitude, over 4.  Each number of a block is rounded to the nearest of +-
    0, 0.5, 1, 1.5, 2, 3, 4, 6 of its scale.  A block with an infinity or a NaN becomes
    NaN.  w may be stored [.., out, in] and passed as its transposed view."""
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [in, out] or [experts, in, out], got {list(w.shape)}")
    dev, stream, code = _start(w, "w", w.dim())
    *lead, n_in, n_out = w.shape
    if w.numel() == 0:
        raise ValueError(f"w must have elements, got {list(w.shape)}")
    layout, w_stride = _weight(w, n_in, n_out)
    blocks = -(-n_in // 32)
    values = _empty((*lead, n_out, 16 * blocks), dtype=_U8, device=dev)
    scales = _empty((*lead, n_out, blocks), dtype=_U8, device=dev)
    experts = lead[0] if lead else 0
    st = _c.load().muon_mx_quantize(code, layout, _int32(experts), n_in, n_out, w.data_ptr(), w_stride,
                                    w.stride(0) if experts > 1 else 0, values.data_ptr(), scales.data_ptr(), stream)
    if st:
        _c.check(st, "muon_mx_quantize")
    return values, scales


def _held(values, scales, dev, n_in=None):
    """(addresses, experts, out) of microscaled weights of n_in steps (any, if None)."""
    if values.dim() not in (2, 3):
        raise ValueError(f"values must be [out, 16 * blocks] or [experts, out, 16 * blocks], got {list(values.shape)}")
    *lead, out, width = values.shape
    if lead and lead[0] == 0:
        raise ValueError(f"values must have experts, got {list(values.shape)}")
    blocks = width // 16 if n_in is None else -(-n_in // 32)
    vp = _contiguous(values, "values", dev, _U8, (*lead, out, 16 * blocks))
    sp = _contiguous(scales, "scales", dev, _U8, (*lead, out, blocks))
    return vp, sp, lead[0] if lead else 0, out


@_operator
def mx_dequantize(values, scales, n_in, dtype=torch.bfloat16):
    """The weights [in, out] or [experts, in, out] that mx_quantize's values and scales
    stand for, rounded to dtype: the transposed view of a contiguous [.., out, in]."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    n_in = int(n_in)
    if n_in < 1:
        raise ValueError(f"n_in must be at least 1, got {n_in}")
    dev, stream = _start_bytes(values)
    vp, sp, experts, out = _held(values, scales, dev, n_in)
    w = _empty((*values.shape[:-1], n_in), dtype=dtype, device=dev)
    st = _c.load().muon_mx_dequantize(_DTYPES[dtype], _int32(experts), n_in, out, vp, sp, w.data_ptr(), stream)
    if st:
        _c.check(st, "muon_mx_dequantize")
    return w.transpose(-1, -2)


def _start_bytes(values):
    """(device index, current stream) of packed values."""
    dev = values.get_device()
    if dev < 0:
        raise ValueError("values must live on a CUDA device")
    if dev != _current_device():
        raise ValueError(f"values is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev, _raw_stream(dev)


def _mx_forward(x, offsets, values, scales, bias, activation, residual):
    dev, stream, code = _start(x, "x", 2)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    rows, n_in = x.shape
    vp, sp, experts, out = _held(values, scales, dev, n_in)
    if (values.dim() == 3) != (offsets is not None):
        raise ValueError(f"values must be [{'experts, ' if offsets is not None else ''}out, 16 * blocks], got "
                         f"{list(values.shape)}")
    off = bp = rp = r_stride = 0
    if offsets is not None:
        off = _contiguous(offsets, "offsets", dev, _I32, (experts + 1,))
    if bias is not None:
        bp = _contiguous(bias, "bias", dev, x.dtype, (out,) if offsets is None else (experts, out))
    if residual is not None:
        _check(residual, "residual", dev, x.dtype, (rows, out))
        rp, r_stride = residual.data_ptr(), _rows(residual, "residual")
    y = _empty((rows, out), dtype=x.dtype, device=dev)
    size = _mx_scratch_size(code, experts, rows, n_in, out)
    ws = _empty(size, dtype=_U8, device=dev) if size else None
    st = _mx_call()(_MX_PACK(code, act, _int32(experts), 0, rows, n_in, out, _rows(x, "x"), r_stride, x.data_ptr(), vp, sp,
                             bp, rp, off, y.data_ptr(), ws.data_ptr() if size else 0, size), stream)
    if st:
        _c.check(st, "muon_mx_linear")
    return y


@_operator
def mx_linear(x, values, scales, bias=None, activation="none", residual=None):
    """act(x' @ w + bias) + residual for weights that mx_quantize packed: x' is x
    [rows, in] rounded to microscaled 4-bit numbers in the same way, row by row.  Sums
    are fp32; bias, residual and the result are of x's type.  Forward only.

    Rounding to 4 bits costs accuracy: normally distributed operands are off by 11.5% each
    (of their norm), the product by 16%."""
    return _mx_forward(x, None, values, scales, bias, activation, residual)


@_operator
def mx_expert_linear(x, offsets, values, scales, bias=None, activation="none", residual=None):
    """mx_linear over an expert tensor: rows offsets[e] .. offsets[e + 1] - 1 of x go
    through values[e], scales[e] and bias[e]; rows of no expert come out zero."""
    return _mx_forward(x, _given(offsets), values, scales, bias, activation, residual)


def check_ops_error() -> None:
    """Synchronises the current device; raises MuonError if a kernel of an
    earlier call gave up a bounded wait."""
    _c.check(_c.load().muon_ops_check_error(), "muon_ops_check_error")
