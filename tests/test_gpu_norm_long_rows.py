"""The layer norm and its gradient over rows of millions of elements against fp64: a
thread adds thousands of them, and a long row keeps the digits of a short one.

The numbers repeat, so that the roundings of one running sum would all go the same way
(1 + 0.98 2^-13 is rounded down each time a sum above 2048 takes it in): its mean
would be off by 6e-5 of itself.  With the roundings of the running sum kept, what is left
are those of a piece's eight elements, two at the end and 15 over the threads: within R =
48 2^-24 of the sum of magnitudes (the squares and products under the sums round three
times more)."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import TINY, U, close, to64

pytestmark = pytest.mark.gpu

R = 48 * 2.0 ** -24
E = 2.0 ** -24


@pytest.mark.parametrize("width", [4 << 20, (4 << 20) + 8, 4000003])
def test_a_long_row(width):
    c = 1 + 0.98 * 2.0 ** -13
    i = torch.arange(width, device="cuda")
    x = (c + torch.where((i // 8) % 2 == 0, 2.0 ** -6, -2.0 ** -6)).float()[None].contiguous()
    dy = (c + torch.where((i // 8) % 4 < 2, 2.0 ** -6, -2.0 ** -6)).float()[None].contiguous()
    w = torch.ones(width, device="cuda")
    for at in (w, None):
        y, mean, rstd = muon.layer_norm(x, at, eps=0.0, keep_stats=True)
        X = to64(x)
        Y, M, S = ref.layer_norm(X, eps=0.0)
        dm = R * abs(X).mean(axis=1)
        close(mean, M, dm + E * abs(M), "mean")
        rel = 0.5 * (R + (dm * S) ** 2) * 1.01 + 4 * E
        close(rstd, S, rel * S, "rstd")
        d = abs(X - M[:, None])
        t = S[:, None] * (dm[:, None] + E * d) + d * S[:, None] * (rel[:, None] + 3 * E) * 1.01 + E * abs(Y)
        close(y, Y, t + U[x.dtype] * (abs(Y) + t) * 1.01 + TINY[x.dtype], "y")
        dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, at, bias=True)
        DY, M, S = to64(dy), to64(mean)[:, None], to64(rstd)[:, None]
        DX, DW, DB = ref.layer_norm_backward(DY, X, M[:, 0], S[:, 0])
        ax, ag = abs((X - M) * S), abs(DY)
        m1, m2 = ag.mean(axis=1, keepdims=True), (ag * ax).mean(axis=1, keepdims=True)
        t = S * (4 * E * ag + (R + 4 * E) * m1 + ax * (R + 8 * E) * m2) * 1.01
        close(dx, DX, t + E * (abs(DX) + t) * 1.01 + TINY[x.dtype], "dx")
        close(dw, DW, 8 * E * ag[0] * ax[0], "dw")
        close(db, DB, E * abs(DB), "db")
    muon.check_ops_error()


def test_infinities_in_a_long_row():
    """The statistics of short rows: an infinite mean, and NaN for both signs."""
    for width in (700, 40000, 40001):
        x = torch.ones(3, width, device="cuda")
        x[0, 5], x[1, 7], x[1, 600], x[2, 3] = float("inf"), float("inf"), -float("inf"), float("nan")
        y, mean, rstd = muon.layer_norm(x, keep_stats=True)
        assert mean[0] == float("inf") and torch.isnan(mean[1:]).all() and torch.isnan(rstd).all() and torch.isnan(y).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_long_row_of_16_bits(dtype):
    """The same bound on rows as a model has them, whole pieces and single elements."""
    for width in (3 << 20, 3000001):
        g = torch.Generator(device="cuda").manual_seed(width)
        x = (torch.randn(2, width, generator=g, device="cuda") * 0.5 + 3).to(dtype)
        _, mean, rstd = muon.layer_norm(x, keep_stats=True)
        X = to64(x)
        _, M, S = ref.layer_norm(X)
        dm = R * abs(X).mean(axis=1)
        close(mean, M, dm + E * abs(M), "mean")
        close(rstd, S, (0.5 * (R + (dm * S) ** 2) * 1.01 + 4 * E) * S, "rstd")
