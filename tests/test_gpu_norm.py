"""The layer norm and its gradient on the GPU against the fp64 oracle, element by
element.

A row's sums take up to 64 additions one after another in a thread and 16 levels
above: within R = 96 2^-24 of the sum of magnitudes.  The mean is off by dm = R mean|x|;
the sum of squares about it by R of itself and dm^2; rstd by half of that, and 4 2^-24
for the quotient, the root and the division."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import TINY, U, acc, close, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
R = 96 * 2.0 ** -24
E = 2.0 ** -24


def _check(x, w, b, eps=1e-5):
    y, mean, rstd = muon.layer_norm(x, w, bias=b, eps=eps, keep_stats=True)
    X = to64(x)
    W = None if w is None else to64(w)
    B = None if b is None else to64(b)
    Y, M, S = ref.layer_norm(X, W, B, eps)
    dm = R * np.abs(X).mean(axis=1)
    close(mean, M, dm + E * np.abs(M), "mean")
    var = 1 / S ** 2 - eps
    rel = 0.5 * (R * var + dm ** 2) * S ** 2 * 1.01 + 4 * E
    close(rstd, S, rel * S, "rstd")
    aw = 1.0 if w is None else np.abs(W)
    D = np.abs(X - M[:, None])
    t = aw * S[:, None] * (dm[:, None] + E * D) + aw * D * S[:, None] * (rel[:, None] + 3 * E) * 1.01
    t = t + E * np.abs(Y) + (0 if b is None else E * np.abs(B))
    close(y, Y, t + U[x.dtype] * (np.abs(Y) + t) * 1.01 + TINY[x.dtype], "y")
    return y, mean, rstd


def _check_backward(dy, x, mean, rstd, w, r, rows_acc=None):
    dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, w, residual=r, bias=True)
    DY, X, M, S = to64(dy), to64(x), to64(mean)[:, None], to64(rstd)[:, None]
    W = np.ones(x.shape[1]) if w is None else to64(w)
    RES = None if r is None else to64(r)
    DX, DW, DB = ref.layer_norm_backward(DY, X, M[:, 0], S[:, 0], W, RES)
    xh = (X - M) * S
    g = DY * W
    ax, ag = np.abs(xh), np.abs(g)
    m1, m2 = ag.mean(axis=1, keepdims=True), (ag * ax).mean(axis=1, keepdims=True)
    # each of g, xh and the two means is rounded, then three operations in a row
    t = S * (4 * E * ag + (R + 4 * E) * m1 + ax * (R + 8 * E) * m2) * 1.01
    if r is not None:
        t = t + E * np.abs(RES)
    dt = x.dtype
    close(dx, DX, t + U[dt] * (np.abs(DX) + t) * 1.01 + TINY[dt], "dx")
    wt = dt if w is None else w.dtype
    a = acc(x.shape[0])
    t = (a + 4 * E) * (np.abs(DY) * ax).sum(axis=0)
    close(dw, DW, t + U[wt] * (np.abs(DW) + t) * 1.01 + TINY[wt], "dw")
    t = a * np.abs(DY).sum(axis=0)
    close(db, DB, t + U[wt] * (np.abs(DB) + t) * 1.01 + TINY[wt], "db")


def _inputs(rows, width, dtype, seed, w_fp32=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    wt = torch.float32 if w_fp32 else dtype
    x = (n(rows, width) * 2 + n(rows, 1)).to(dtype)
    return x, (1 + 0.3 * n(width)).to(wt), (0.2 * n(width)).to(wt), n(rows, width).to(dtype), n(rows, width).to(dtype)


# a row in a few lanes, a warp, a block with 16 or 32 elements a thread, in none; whole pieces and ragged
CASES = [(1, 1), (3, 2), (5, 8), (70, 31), (9, 64), (33, 200), (40, 512), (6, 513), (10, 520), (7, 1000), (5, 1001),
         (700, 1024), (3, 4096), (5, 4104), (2, 6000), (4, 8192), (3, 8191), (2, 8200), (2, 16384), (2, 16392), (3, 20001),
         (1, 40000)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_layer_norm(case, dtype):
    rows, width = case
    for w_fp32 in (False, True):
        x, w, b, dy, r = _inputs(rows, width, DT[dtype], rows + width, w_fp32)
        _, mean, rstd = _check(x, w, b)
        _check_backward(dy, x, mean, rstd, w, r)
    _, mean, rstd = _check(x, None, None)
    _check_backward(dy, x, mean, rstd, None, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(5000, 4096), (1300, 48), (2600, 777), (400, 9000)])
def test_many_rows(rows, width, dtype):
    """Blocks that work through many rows, and sums over all of them."""
    x, w, b, dy, r = _inputs(rows, width, DT[dtype], 7)
    _, mean, rstd = _check(x, w, b)
    _check_backward(dy, x, mean, rstd, w, r)


def test_each_gradient_alone_is_the_same():
    x, w, b, dy, r = _inputs(300, 1024, torch.bfloat16, 3)
    _, mean, rstd = muon.layer_norm(x, w, bias=b, keep_stats=True)
    dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    assert muon.layer_norm_backward(dy, x, mean, rstd, w, dw=False)[1:] == (None, None)
    assert torch.equal(muon.layer_norm_backward(dy, x, mean, rstd, w, dw=False)[0], dx)
    assert torch.equal(muon.layer_norm_backward(dy, x, mean, rstd, w, dx=False)[1], dw)
    only = muon.layer_norm_backward(dy, x, mean, rstd, w, dx=False, dw=False, bias=True)
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)
    for _ in range(3):  # and every time
        assert all(torch.equal(p, q) for p, q in zip(muon.layer_norm_backward(dy, x, mean, rstd, w, bias=True), (dx, dw, db)))
    assert torch.equal(muon.layer_norm(x, w, bias=b), muon.layer_norm(x, w, bias=b, keep_stats=True)[0])


@pytest.mark.parametrize("width", [56, 1024, 4096, 10000])
def test_rows_do_not_depend_on_their_batch(width):
    x, w, b, dy, _ = _inputs(1000, width, torch.bfloat16, 4)
    y, mean, rstd = muon.layer_norm(x, w, bias=b, keep_stats=True)
    dx, _, _ = muon.layer_norm_backward(dy, x, mean, rstd, w)
    pick = slice(400, 403)
    dx2, _, _ = muon.layer_norm_backward(dy[pick], x[pick], mean[pick], rstd[pick], w)
    assert torch.equal(dx[pick], dx2)
    # (few rows and many may take other numbers of threads, and other orders of a row's sums)
    _check(x[pick], w, b)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,width", [(1200, 700), (700, 4097), (400, 9001), (330, 16383)])
def test_rows_between_boundaries(rows, width, dtype):
    """Rows that start and end anywhere, each tensor's elsewhere, many to a block."""
    dt = DT[dtype]
    x, w, b, dy, r = _inputs(rows, width, dt, 8)

    def within(t, lead, more):
        wide = torch.full((rows, width + more), float("nan"), dtype=dt, device="cuda")
        wide[:, lead:lead + width] = t
        return wide[:, lead:lead + width]

    x, dy, r = within(x, 3, 7), within(dy, 1, 1), within(r, 0, 4)
    _, mean, rstd = _check(x, w, b)
    _check_backward(dy, x, mean, rstd, w, r)


def test_large_and_small_rows():
    """Means far above the spread, tiny and constant rows, the largest numbers."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(6, 512, generator=g, device="cuda")
    x[1] += 1000.0
    x[2] *= 1e-12
    x[3] = 3.0
    x[4] *= 1e15
    x[5] = 0.0
    _, mean, rstd = _check(x, None, None)
    dy = torch.randn(6, 512, generator=g, device="cuda")
    _check_backward(dy[:3], x[:3], mean[:3], rstd[:3], None, None)
    y = muon.layer_norm(x[3:4].contiguous(), eps=0.0)
    assert torch.isnan(y).all()  # 0 times infinity, as the formula has it


def test_non_finite_rows_stay_alone():
    x, w, b, dy, _ = _inputs(40, 700, torch.bfloat16, 6)
    clean = muon.layer_norm(x, w, bias=b, keep_stats=True)
    bad = x.clone()
    bad[7, 3], bad[21, 699] = math.nan, math.inf
    y, mean, rstd = muon.layer_norm(bad, w, bias=b, keep_stats=True)
    keep = [i for i in range(40) if i not in (7, 21)]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(mean[keep], clean[1][keep])
    assert torch.isnan(y[7]).all() and torch.isnan(y[21]).all()
    dx, dw, _ = muon.layer_norm_backward(dy, bad, mean, rstd, w)
    want, _, _ = muon.layer_norm_backward(dy, x, clean[1], clean[2], w)
    assert torch.equal(dx[keep], want[keep]) and torch.isnan(dx[7]).all() and torch.isnan(dw).all()


@pytest.mark.parametrize("shift", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_alignment(dtype, shift):
    x, w, b, dy, r = _inputs(33, 1100, DT[dtype], 8)
    part = slice(shift, shift + 1024)
    y, mean, rstd = _check(x[:, part], w[part], b[part].clone())
    _check_backward(dy[:, part], x[:, part], mean, rstd, w[part], r[:, part])
    one = x[4:5, part]  # a single row of any pitch
    _check(one, None, None)


def test_no_rows_streams_and_graphs():
    x, w, b, dy, r = _inputs(50, 264, torch.float16, 9)
    y, mean, rstd = muon.layer_norm(x[:0], w, bias=b, keep_stats=True)
    assert y.shape == (0, 264) and mean.shape == (0,)
    dx, dw, db = muon.layer_norm_backward(dy[:0], x[:0], mean, rstd, w, bias=True)
    assert dx.shape == (0, 264) and not dw.any() and not db.any()
    want = muon.layer_norm(x, w, bias=b, keep_stats=True)
    grads = muon.layer_norm_backward(dy, x, *want[1:], w, residual=r, bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = muon.layer_norm(x, w, bias=b, keep_stats=True, stream=s)
    back = muon.layer_norm_backward(dy, x, got[1], got[2], w, residual=r, bias=True, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got, *back), (*want, *grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = muon.layer_norm(x, w, bias=b, keep_stats=True)
        held += muon.layer_norm_backward(dy, x, held[1], held[2], w, residual=r, bias=True)
    for i in range(3):
        x.copy_(torch.roll(x, 1, 0))
        graph.replay()
        fresh = muon.layer_norm(x, w, bias=b, keep_stats=True)
        fresh += muon.layer_norm_backward(dy, x, fresh[1], fresh[2], w, residual=r, bias=True)
        assert all(torch.equal(p, q) for p, q in zip(held, fresh)), i
    muon.check_ops_error()


def test_gradient_matches_differences():
    """Central differences of the fp32 result along random directions, in 64 bits outside:
    off by h^2 f''' / 6 and by the rows' errors over h."""
    g = torch.Generator(device="cuda").manual_seed(10)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, b, dy, d = n(20, 96), n(96), n(96), n(20, 96), n(20, 96)
    _, mean, rstd = muon.layer_norm(x, w, bias=b, keep_stats=True)
    dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    h = 1e-2
    f = lambda x, w, b: (muon.layer_norm(x, w, bias=b).double() * dy.double()).sum(1)  # noqa: E731
    num = (f(x + h * d, w, b) - f(x - h * d, w, b)) / (2 * h)
    got = (dx.double() * d.double()).sum(1)
    # rows of 96: |f'''| below 100 |d|^3 / sqrt(96)^2 ~ 1e3: 1e-4 / 6 * 1e3 = 2e-2; rounding 96 * 2^-22 * 4 / h = 1e-2
    assert ((num - got).abs() < 3e-2).all()
    v = n(96)
    num = (f(x, w + h * v, b) - f(x, w - h * v, b)).sum() / (2 * h)  # linear in w and b
    assert abs(float(num - (dw.double() * v.double()).sum())) < 2e-2
    num = (f(x, w, b + h * v) - f(x, w, b - h * v)).sum() / (2 * h)
    assert abs(float(num - (db.double() * v.double()).sum())) < 2e-2


def test_refusals():
    x, w, b, dy, r = _inputs(4, 16, torch.float32, 1)
    _, mean, rstd = muon.layer_norm(x, w, keep_stats=True)
    for f in (lambda: muon.layer_norm(x[0]), lambda: muon.layer_norm(x.double()), lambda: muon.layer_norm(x.t()),
              lambda: muon.layer_norm(x, w.half()), lambda: muon.layer_norm(x, w[:8]), lambda: muon.layer_norm(x, w.cpu()),
              lambda: muon.layer_norm(x.half(), w.half(), bias=b), lambda: muon.layer_norm(x, w, bias=b[:3]),
              lambda: muon.layer_norm(x, w[::2]), lambda: muon.layer_norm_backward(dy.half(), x, mean, rstd, w),
              lambda: muon.layer_norm_backward(dy, x, mean[:2], rstd, w),
              lambda: muon.layer_norm_backward(dy, x, mean, rstd.double(), w),
              lambda: muon.layer_norm_backward(dy, x, mean, rstd, w, residual=r[:2]),
              lambda: muon.layer_norm_backward(dy, x, mean, rstd, w, residual=r, dx=False),
              lambda: muon.layer_norm_backward(dy, x, mean, rstd, w, dx=False, dw=False)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(muon.MuonError):
        muon.layer_norm(x, w, eps=-1.0)
    with pytest.raises(muon.MuonError):
        muon.layer_norm(x[:, :0])
