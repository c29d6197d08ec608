"""A layer's product with its epilogue, dense and per expert, and its gradient
on the GPU against the fp64 oracle, element by element: types, both weight
orders, one row to hundreds, odd widths, row strides, unaligned bases, empty
experts, rows of no expert, non-finite rows next to finite ones, guard bands,
streams, graphs and repeatability."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from newton_schulz_bucket_gb300 import _capi

from layers_tol import check_backward, check_forward

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _problem(rows, n_in, n_out, dtype, seed, experts=0, out_in=False):
    g = _gen(seed)
    lead = (experts,) if experts else ()
    x = _normal(g, rows, n_in, dtype=dtype)
    shape = (*lead, n_out, n_in) if out_in else (*lead, n_in, n_out)
    w = _normal(g, *shape, std=n_in ** -0.5, dtype=dtype)
    w = w.transpose(-1, -2) if out_in else w
    b = _normal(g, *lead, n_out, std=0.3, dtype=dtype)
    r = _normal(g, rows, n_out, dtype=dtype)
    dy = _normal(g, rows, n_out, std=0.1, dtype=dtype)
    z = _normal(g, rows, n_out, std=1.5, dtype=dtype)
    return x, w, b, r, dy, z


def _both(rows, n_in, n_out, dtype, act, out_in, seed, offsets=None, bias=True, residual=True):
    experts = 0 if offsets is None else len(offsets) - 1
    x, w, b, r, dy, z = _problem(rows, n_in, n_out, dtype, seed, experts, out_in)
    b, r = (b if bias else None), (r if residual else None)
    if offsets is None:
        y, zz = muon.linear(x, w, bias=b, activation=act, residual=r, keep_preact=True)
        got = muon.linear_backward(dy, x, w, preact=z, activation=act, bias=True)
    else:
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        y, zz = muon.expert_linear(x, off, w, bias=b, activation=act, residual=r, keep_preact=True)
        got = muon.expert_linear_backward(dy, x, off, w, preact=z, activation=act, bias=True)
    muon.check_ops_error()
    if min(n_in, n_out) > 1:  # w's memory order
        assert got[1].stride() == w.stride()
    check_forward(y, zz, x, w, b, act, r, offsets)
    check_backward(got, dy, x, w, z, act, offsets)


SIZES = [(1, 1, 1), (1, 64, 128), (1, 512, 300), (2, 100, 8), (7, 65, 63), (16, 256, 264), (17, 1000, 136),
         (33, 128, 520), (64, 320, 257), (100, 72, 1), (129, 1, 200), (130, 192, 384), (200, 333, 130),
         (256, 512, 512), (257, 264, 1032), (300, 1033, 96), (515, 640, 768), (700, 136, 513)]


@pytest.mark.parametrize("out_in", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_dense(size, dtype, out_in):
    act = ACTS[(sum(size) + out_in) % len(ACTS)]
    _both(*size, DT[dtype], act, out_in, seed=sum(size))


@pytest.mark.parametrize("out_in", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("size", [(1, 4097, 515), (5, 2051, 1025), (16, 66, 9000), (40, 515, 130), (63, 777, 2049),
                                  (64, 9001, 40)], ids=lambda s: "x".join(map(str, s)))
def test_few_rows_of_odd_widths(size, out_in):
    """Long sums shared by a cluster, rows that start on no 16 bytes."""
    _both(*size, torch.bfloat16, "silu", out_in, seed=sum(size))
    x, w, b, r, dy, z = _problem(*size, torch.float16, 3, out_in=out_in)
    check_forward(muon.linear(x, w), None, x, w, None, "none", None)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [5, 384])
def test_activations(rows, dtype, act):
    _both(rows, 192, 320, DT[dtype], act, False, seed=11, bias=False, residual=False)


OFFSETS = {
    "even": [0, 64, 128, 192, 256],
    "ragged": [0, 1, 1, 70, 199, 200, 263, 500],
    "one_takes_all": [0, 0, 0, 300, 300],
    "few_rows": [0, 0, 1, 1, 1, 3, 3, 4, 4, 5],
    "unowned": [0, 3, 60, 60, 171],
    "none": [0, 0, 0],
    "large": [0, 513, 600, 600, 1000],
}


@pytest.mark.parametrize("out_in", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("widths", [(64, 128), (200, 272), (97, 131), (520, 256)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", list(OFFSETS))
def test_experts(kind, widths, dtype, out_in):
    off = OFFSETS[kind]
    rows = off[-1] + (37 if kind in ("unowned", "none") else 0)
    act = ACTS[(len(off) + widths[0]) % len(ACTS)]
    _both(rows, *widths, DT[dtype], act, out_in, seed=len(off), offsets=off)


def test_many_experts():
    g = np.random.default_rng(5)
    off = np.concatenate([[0], np.cumsum(g.integers(0, 3, 1024))]).tolist()
    _both(off[-1], 64, 72, torch.bfloat16, "silu", False, seed=6, offsets=off)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_experts_keep_to_themselves(dtype):
    """Non-finite rows of one expert, and of none, reach no other expert's
    outputs and gradients."""
    off = [0, 70, 133, 133, 200]
    x, w, b, r, dy, z = _problem(230, 192, 136, DT[dtype], 3, 4)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    want = muon.expert_linear(x, o, w, bias=b, activation="silu")
    dwant = muon.expert_linear_backward(dy, x, o, w, preact=z, activation="silu", bias=True)
    x2, dy2, z2 = x.clone(), dy.clone(), z.clone()
    for t in (x2, dy2, z2):
        t[70:133:2] = math.nan
        t[71:133:2] = math.inf
        t[200:] = math.nan
    got = muon.expert_linear(x2, o, w, bias=b, activation="silu")
    dgot = muon.expert_linear_backward(dy2, x2, o, w, preact=z2, activation="silu", bias=True)
    keep = torch.ones(230, dtype=torch.bool, device="cuda")
    keep[70:133] = False
    assert torch.equal(got[keep], want[keep]) and torch.equal(dgot[0][keep], dwant[0][keep])
    assert not got[200:].any() and not dgot[0][200:].any()
    others = [0, 2, 3]
    assert torch.equal(dgot[1][others], dwant[1][others]) and torch.equal(dgot[2][others], dwant[2][others])
    assert torch.isnan(dgot[1][1]).any()


@pytest.mark.parametrize("dtype", list(DT))
def test_non_finite_values_follow_the_formula(dtype):
    x, w, b, r, dy, z = _problem(40, 128, 136, DT[dtype], 4)
    x[3, 5], x[9, 0] = math.nan, math.inf
    y = muon.linear(x, w, bias=b, activation="relu")
    assert torch.isnan(y[3]).all()
    assert not torch.isfinite(y[9]).logical_and(w[0] > 0).any()
    assert torch.isfinite(y[[0, 1, 2, 4, 8, 10]]).all()


@pytest.mark.parametrize("experts", [0, 3])
@pytest.mark.parametrize("dtype", list(DT))
def test_no_rows(dtype, experts):
    x, w, b, r, dy, z = _problem(0, 48, 40, DT[dtype], 1, experts)
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    if experts:
        y = muon.expert_linear(x, off, w, bias=b)
        dx, dw, db = muon.expert_linear_backward(dy, x, off, w, bias=True)
    else:
        y = muon.linear(x, w, bias=b)
        dx, dw, db = muon.linear_backward(dy, x, w, bias=True)
    assert y.shape == (0, 40) and dx.shape == (0, 48)
    assert dw.shape == w.shape and not dw.any() and not db.any()


@pytest.mark.parametrize("rows", [3, 90, 400])
@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_unaligned_bases(dtype, rows):
    """Column slices of wider tensors (every tensor at an odd element offset)
    give the bits of contiguous copies' values within the bounds."""
    dt, g = DT[dtype], _gen(8)
    x = _normal(g, rows, 300, dtype=dt)[:, 3:203]
    w = _normal(g, 210, 400, std=0.07, dtype=dt)[5:205, 1:265]
    r = _normal(g, rows, 500, dtype=dt)[:, 7:271]
    dy = _normal(g, rows, 270, std=0.1, dtype=dt)[:, 1:265]
    b = _normal(g, 300, dtype=dt)[1:265]
    z = _normal(g, rows * 264 + 1, dtype=dt)[1:].view(rows, 264)
    y, zz = muon.linear(x, w, bias=b, activation="gelu", residual=r, keep_preact=True)
    check_forward(y, zz, x, w, b, "gelu", r)
    got = muon.linear_backward(dy, x, w, preact=z, activation="gelu", bias=True)
    check_backward(got, dy, x, w, z, "gelu")
    we = _normal(g, 3, 210, 400, std=0.07, dtype=dt)[:, 5:205, 1:265]
    off = [0, rows // 3, rows // 3, rows]
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    y = muon.expert_linear(x, o, we, residual=r)
    check_forward(y, None, x, we, None, "none", r, off)
    check_backward(muon.expert_linear_backward(dy, x, o, we, bias=True), dy, x, we, None, "none", off)


@pytest.mark.parametrize("parts", [dict(dx=True, dw=False), dict(dx=False, dw=True), dict(dx=False, dw=False, bias=True)])
def test_parts_of_the_gradient(parts):
    x, w, b, r, dy, z = _problem(70, 128, 192, torch.bfloat16, 2)
    full = muon.linear_backward(dy, x, w, preact=z, activation="silu", bias=True)
    got = muon.linear_backward(dy, x, w, preact=z, activation="silu", **parts)
    want = [parts.get("dx", True), parts.get("dw", True), parts.get("bias", False)]
    for a, f, on in zip(got, full, want):
        assert (a is not None) == on and (not on or torch.equal(a, f))


@pytest.mark.parametrize("rows,n_in,n_out", [(3, 1024, 512), (100, 2048, 256), (300, 4096, 264), (600, 320, 512)])
def test_same_bits_every_time(rows, n_in, n_out):
    x, w, b, r, dy, z = _problem(rows, n_in, n_out, torch.bfloat16, 9)
    first = (muon.linear(x, w, bias=b), *muon.linear_backward(dy, x, w, preact=z, activation="gelu", bias=True))
    for _ in range(3):
        again = (muon.linear(x, w, bias=b), *muon.linear_backward(dy, x, w, preact=z, activation="gelu", bias=True))
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_side_stream_and_graph():
    x, w, b, r, dy, z = _problem(200, 256, 320, torch.bfloat16, 10)
    want = muon.linear(x, w, bias=b, activation="silu")
    dwant = muon.linear_backward(dy, x, w, preact=z, activation="silu", bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = muon.linear(x, w, bias=b, activation="silu", stream=s)
    dgot = muon.linear_backward(dy, x, w, preact=z, activation="silu", bias=True, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(p, q) for p, q in zip(dgot, dwant))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = muon.linear(x, w, bias=b, activation="silu")
        d = muon.linear_backward(dy, x, w, preact=z, activation="silu", bias=True)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, muon.linear(x, w, bias=b, activation="silu"))
    again = muon.linear_backward(dy, x, w, preact=z, activation="silu", bias=True)
    assert all(torch.equal(p, q) for p, q in zip(d, again))


def test_graph_that_forks_and_joins():
    """Calls on two streams inside one capture, each starting from the other's
    result, next to PyTorch's own kernels and a memset."""
    x, w, b, r, dy, z = _problem(160, 256, 256, torch.bfloat16, 20)
    w2 = _normal(_gen(21), 256, 256, std=1 / 16, dtype=torch.bfloat16)

    def run(side):
        main = torch.cuda.current_stream()
        a = muon.linear(x, w, activation="silu")
        if side is not None:
            side.wait_stream(main)
        c = muon.linear(a, w2, stream=side) if side is not None else muon.linear(a, w2)
        d = muon.linear(a, w, activation="relu")
        zero = torch.zeros_like(d)
        if side is not None:
            main.wait_stream(side)
        e = muon.linear(c + zero, w, residual=d)
        g = muon.linear_backward(e, c, w2, bias=True)
        return a, c, d, e, *g

    want = run(None)
    side = torch.cuda.Stream()
    eager = run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(eager, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want))


PAD = 512


def _guarded(n, dtype):
    back = torch.full((n + 2 * PAD,), -77.0, dtype=dtype, device="cuda")
    return back, back[PAD:PAD + n]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,n_in,n_out,experts", [(5, 130, 72, 0), (150, 72, 264, 0), (301, 264, 137, 0),
                                                     (40, 96, 130, 5), (333, 136, 264, 3)])
def test_guard_bands(rows, n_in, n_out, experts, dtype):
    """No output, and not the workspace, is written outside its own bytes."""
    dt = DT[dtype]
    x, w, b, r, dy, z = _problem(rows, n_in, n_out, dt, 12, experts)
    mats = max(experts, 1)
    outs = {k: _guarded(n, dt) for k, n in (("y", rows * n_out), ("preact_out", rows * n_out), ("dx", rows * n_in),
                                            ("dw", mats * n_in * n_out), ("db", mats * n_out))}
    a = _capi.muon_linear_args()
    a.dtype, a.activation, a.experts = {"bf16": 2, "fp32": 0}[dtype], 2, experts
    a.rows, a.out = rows, n_out
    setattr(a, "in", n_in)
    a.x_stride, a.w_stride, a.w_expert_stride, a.residual_stride, a.dy_stride = n_in, n_out, n_in * n_out, n_out, n_out
    a.x, a.w, a.bias, a.residual, a.dy, a.preact = (t.data_ptr() for t in (x, w, b, r, dy, z))
    off = torch.linspace(0, rows, experts + 1, device="cuda").int()
    a.offsets = off.data_ptr()
    for k, (back, v) in outs.items():
        setattr(a, k, v.data_ptr())
    L = _capi.load()
    st = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    for backward, call in ((0, L.muon_linear), (1, L.muon_linear_backward)):
        n = C.c_size_t()
        assert L.muon_linear_workspace(C.byref(a), backward, C.byref(n)) == 0
        ws = torch.full((n.value + 1024,), 0x5a, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), n.value
        assert call(C.byref(a), st) == 0, L.muon_last_error()
        torch.cuda.synchronize()
        assert (ws[n.value:] == 0x5a).all()
    for k, (back, v) in outs.items():
        assert (back[:PAD] == -77).all() and (back[PAD + v.numel():] == -77).all(), k
        assert torch.isfinite(v).all() and not (v == -77).all(), k
    muon.check_ops_error()


def test_offsets_out_of_range_are_clamped():
    """Offsets that point outside the rows read and write nothing outside."""
    x, w, b, r, dy, z = _problem(64, 64, 64, torch.bfloat16, 13, 3)
    off = torch.tensor([0, 50, 1 << 30, 1 << 30], dtype=torch.int32, device="cuda")
    y = muon.expert_linear(x, off, w)
    check_forward(y, None, x, w, None, "none", None, [0, 50, 64, 64])
    check_backward(muon.expert_linear_backward(dy, x, off, w, bias=True), dy, x, w, None, "none", [0, 50, 64, 64])


def test_gradient_matches_differences():
    """Central differences of the fp32 forward pass itself, along random
    directions: with step h the quotient is off by h^2 f''' / 6 and by the
    forward pass's rounding over h."""
    off = [0, 9, 9, 30]
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w, b, r, dy, _ = _problem(30, 24, 20, torch.float32, 14, 3)
    _, z = muon.expert_linear(x, o, w, bias=b, activation="gelu_tanh", keep_preact=True)
    dx, dw, db = muon.expert_linear_backward(dy, x, o, w, preact=z, activation="gelu_tanh", bias=True)
    h, g = 1e-2, _gen(15)

    def f(xx, ww, bb):
        return (muon.expert_linear(xx, o, ww, bias=bb, activation="gelu_tanh").double() * dy.double()).sum().item()

    for i, grad in enumerate((dx, dw, db)):
        args = [x, w, b]
        d = torch.randn(args[i].shape, generator=g, device="cuda") * 0.1
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * d, args[i] - h * d
        num = (f(*hi) - f(*lo)) / (2 * h)
        got = (grad.double() * d.double()).sum().item()
        # 600 values of dy ~ 0.1, y ~ 1 with rounding 2^-22 each: 600 * 0.1 * 2^-22 / h = 1.4e-3;
        # third derivative of the sum along d below 10: 1e-4 * 10 / 6 = 1.7e-4
        assert abs(num - got) < 2e-3, (i, num, got)


def test_refusals():
    x, w, b, r, dy, z = _problem(8, 16, 24, torch.bfloat16, 16)
    bad = [lambda: muon.linear(x.cpu(), w), lambda: muon.linear(x, w.float()), lambda: muon.linear(x, w[:8]),
           lambda: muon.linear(x[0], w), lambda: muon.linear(x, w, activation="tanh"),
           lambda: muon.linear(x, w, bias=b[:3]), lambda: muon.linear(x, w, residual=r[:, :8]),
           lambda: muon.linear(x.double(), w.double()), lambda: muon.linear(x[:, ::2], w[::2]),
           lambda: muon.linear(x[:1].expand(8, 16), w), lambda: muon.linear_backward(dy, x, w, activation="silu"),
           lambda: muon.linear_backward(dy, x, w, dx=False, dw=False),
           lambda: muon.linear_backward(dy, x, w, preact=z.t().contiguous().t(), activation="silu"),
           lambda: muon.expert_linear(x, None, w[None]),
           lambda: muon.expert_linear(x, torch.zeros(2, dtype=torch.int64, device="cuda"), w[None]),
           lambda: muon.expert_linear(x, torch.zeros(3, dtype=torch.int32, device="cuda"), w[None])]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def _check_dw(dw, x, dz, offsets):
    """dw of 16-bit x and dz (no activation) against fp64 products on the GPU,
    expert by expert: sums of fp32 terms, rounded once."""
    from layers_tol import TINY, U, acc
    dt = x.dtype
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        a, b = x[lo:hi].double(), dz[lo:hi].double()
        want, size = a.T @ b, a.abs().T @ b.abs()
        tol = acc(hi - lo) * size
        tol += U[dt] * (want.abs() + tol) * 1.01 + TINY[dt]
        bad = (dw[e].double() - want).abs() > tol
        assert not bad.any(), f"expert {e} ({hi - lo} rows): {int(bad.sum())} of {bad.numel()} off"


@pytest.mark.parametrize("out_in", [False, True], ids=["in_out", "out_in"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weight_gradients_of_many_tiles(dtype, out_in):
    """More tiles than the GPU takes at a time: empty experts, sums that end on and
    beside a block of 64, and rows of NaN that belong to none."""
    g = np.random.default_rng(8)
    counts = g.integers(0, 200, 128)
    counts[[0, 5, 6, 127]] = 0
    counts[[1, 2, 3, 9, 64, 126]] = [384, 385, 383, 700, 64, 1]
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    rows = off[-1] + 11
    x, w, b, r, dy, z = _problem(rows, 264, 2000, DT[dtype], 17, 1, out_in)
    w = w.expand(128, *w.shape[1:]).contiguous() if not out_in else w.transpose(1, 2).expand(128, 2000, 264).contiguous().transpose(1, 2)
    x[off[-1]:] = math.nan
    dy[off[-1]:] = math.nan
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    for _ in range(2):
        dx, dw, db = muon.expert_linear_backward(dy, x, o, w, dx=False)
        muon.check_ops_error()
        _check_dw(dw, x, dy, off)


def test_many_experts_keep_apart():
    """NaN rows of every fourth expert reach no other expert's weight gradient."""
    counts = np.tile([100, 37, 300, 64], 32)
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    x, w, b, r, dy, z = _problem(off[-1], 256, 2048, torch.bfloat16, 18)
    w = torch.zeros(128, 256, 2048, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    want = muon.expert_linear_backward(dy, x, o, w, dx=False)[1]
    _check_dw(want, x, dy, off)
    for e in range(1, 128, 4):
        x[off[e]:off[e + 1]] = math.nan
        dy[off[e]:off[e + 1]] = math.inf
    got = muon.expert_linear_backward(dy, x, o, w, dx=False)[1]
    keep = [e for e in range(128) if e % 4 != 1]
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[1::4]).all()


@pytest.mark.parametrize("rows", [70, 300, 384, 385])
def test_weight_gradient_of_a_large_matrix(rows):
    """A matrix of more tiles than the GPU takes at a time, odd widths, short sums."""
    x, w, b, r, dy, z = _problem(rows, 4100, 16000, torch.bfloat16, 19)
    dw = muon.linear_backward(dy, x, w, dx=False)[1]
    muon.check_ops_error()
    _check_dw(dw[None], x, dy, [0, rows])
