"""The layer products at the ends of their range: tails of the activations,
pre-activations near the type's largest value, the worst mantissas and the
non-finite values of fp32 operands, very long sums and very wide matrices."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

from layers_tol import TINY, U, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SMOOTH = ["silu", "gelu", "gelu_tanh"]


def _tail(z, kind):
    """(act(z), act'(z), a bound of their relative error in fp32) for z <= -3,
    without the cancellation that 1 + erf or 1 + tanh has there."""
    phi = np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu":
        # erfc: 4 ulp of its own; its argument is off by 1.5 roundings of 2^-24, which
        # z^2 + 1 magnifies; the exponential of z^2 / 2 likewise, and its own error
        # grows by 1.2 ulp a unit of its argument
        cdf = np.array([math.erfc(-v / math.sqrt(2)) / 2 for v in z])
        return z * cdf, cdf + z * phi, 2 * z * z + 16
    if kind == "silu":
        w, dw = z, np.ones_like(z)
    else:
        w = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        dw = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + np.exp(-w))
    # w is off by 6 roundings of 2^-24 at most, the exponential by 2 + 1.2 |w| ulp
    return z * p, p + z * p * (1 - p) * dw, 5 * np.abs(w) + 24


@pytest.mark.parametrize("kind", SMOOTH)
@pytest.mark.parametrize("dtype", list(DT))
def test_activation_tails_keep_their_relative_error(dtype, kind):
    """z in [-9, -3], through a 1 x 1 weight of 1 (products are exact).  The slope
    adds two terms of opposite sign of which the larger is at most 1.6 times the
    sum there."""
    dt = DT[dtype]
    z = torch.linspace(-9, -3, 400, device="cuda").to(dt)[:, None].contiguous()
    one = torch.ones(1, 1, dtype=dt, device="cuda")
    y = muon.linear(z, one, activation=kind)
    dx = muon.linear_backward(torch.ones_like(z), z, one, preact=z, activation=kind, dw=False)[0]
    muon.check_ops_error()
    want, slope, rel = _tail(to64(z)[:, 0], kind)
    for what, got, ref, r in (("y", y, want, rel * 2.0 ** -23), ("dx", dx, slope, 2.6 * rel * 2.0 ** -23)):
        err = np.abs(to64(got)[:, 0] - ref)
        tol = (r + 1.01 * U[dt]) * np.abs(ref) + TINY[dt]
        assert (err <= tol).all(), f"{what}: {np.max(err / np.abs(ref)):.3g} of the value, allowed {np.max(r):.3g}"


@pytest.mark.parametrize("kind", ["relu", *SMOOTH])
@pytest.mark.parametrize("dtype", list(DT))
def test_slopes_of_large_preactivations(dtype, kind):
    """Finite pre-activations of any size: the value is z or 0, the slope 1 or 0."""
    dt = DT[dtype]
    most = float(torch.finfo(dt).max)
    z = [v for v in (100.0, 1e4, 1e10, 1.9e19, 5e19, 1e20, 1e30, most / 2, most) if v <= most]
    z = torch.tensor([*z, *(-v for v in z)], dtype=torch.float64, device="cuda").to(dt)[:, None]
    one = torch.ones(1, 1, dtype=dt, device="cuda")
    up = (z > 0).to(dt)
    dx, dw, db = muon.linear_backward(torch.ones_like(z), torch.ones_like(z), one, preact=z, activation=kind, bias=True)
    assert torch.equal(dx, up)
    assert dw.item() == db.item() == up.sum().item()
    assert torch.equal(muon.linear(z, one, activation=kind), z * up)


@pytest.mark.parametrize("rows", [8, 300])
def test_fp32_products_of_the_worst_mantissas(rows):
    """One-term sums to within 2^-22 of the product, as the header states: of
    numbers whose three parts are all as large as they can be, and of any.
    (Left-out partial products 2^-24, one truncating add at the product's size
    2^-23, the adds of the smaller ones below 2^-29.)"""
    g = np.random.default_rng(3)
    bits = np.concatenate([np.array([0x3f80ffff, 0x3f80fffe, 0x3f80feff, 0x3f807fff, 0x3f808000, 0x3f808001, 0x3f80ff7f,
                                     0x3fffffff, 0x3f817f7f], dtype=np.uint32),
                           g.integers(0x3f800000, 0x40000000, 400, dtype=np.uint32),
                           0x3f800000 + (g.integers(0, 128, 400, dtype=np.uint32) << 16) + g.integers(0xff00, 0x10000, 400, dtype=np.uint32)])
    a = bits.view(np.float32).astype(np.float64)
    x, w = np.resize(a, rows), a * np.where(np.arange(a.size) % 3 == 0, -2.0 ** 20, 2.0 ** -30)
    y = muon.linear(torch.tensor(x, dtype=torch.float32, device="cuda")[:, None],
                    torch.tensor(w, dtype=torch.float32, device="cuda")[None])
    want = x[:, None] * w
    rel = np.abs(to64(y) - want) / np.abs(want)
    assert rel.max() <= 2.0 ** -22, rel.max() * 2.0 ** 22


def test_fp32_products_next_to_the_largest_number():
    """Operands that rounding to fewer bits would carry past the largest number."""
    most = float(np.finfo(np.float32).max)
    x = torch.tensor([[most], [-most], [most * (1 - 2.0 ** -10)], [3.3961775e38]], device="cuda")
    w = torch.tensor([[0.25, -0.4999, 1e-30, 2.0 ** -40]], device="cuda")
    want = to64(x) * to64(w)
    assert (np.abs(to64(muon.linear(x, w)) - want) <= 2.0 ** -22 * np.abs(want)).all()


def _same(got, want, tol):
    """Infinities and NaN where the formula has them, finite values within tol."""
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isposinf(got), torch.isposinf(want))
    assert torch.equal(torch.isneginf(got), torch.isneginf(want))
    live = torch.isfinite(want)
    assert ((got - want).abs()[live] <= tol).all()


@pytest.mark.parametrize("n", [130, 1024])
@pytest.mark.parametrize("rows", [6, 40, 200])
def test_fp32_infinities_follow_the_formula(rows, n):
    """An infinity in either operand, against weights that fill 8, 16 and 24 bits,
    zeros, infinities of both signs and NaN; forward, both gradients, and
    through experts.  Finite sums: 96 terms of size 4."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    k, inf = 96, math.inf
    x = torch.randn(rows, k, generator=g, device="cuda")
    w = torch.randn(k, n, generator=g, device="cuda")
    w[3, :8] = torch.tensor([1.0, -1.0, 0.5, 1.0 + 2.0 ** -12, 0.1, -0.1, 0.0, -0.0])
    w[3, 8:11] = torch.tensor([inf, -inf, math.nan])
    w[60, 20], w[61, 20], w[62, 21] = inf, -inf, -inf
    x[0, 3], x[1, 3], x[2, 60], x[3, 5] = inf, -inf, inf, math.nan
    x[4, 3], x[4, 60] = inf, -inf
    x[5, 62] = 0.0
    dy = torch.randn(rows, n, generator=g, device="cuda")
    dy[rows - 1, 4], dy[0, 2], dy[1, 1] = inf, -inf, math.nan
    tol = (1024 + 16) * 2.0 ** -23 * 16 * n
    d = [t.double().cpu() for t in (x, w, dy)]
    _same(muon.linear(x, w), d[0] @ d[1], tol)
    dx, dw, _ = muon.linear_backward(dy, x, w)
    _same(dx, d[2] @ d[1].T, tol)
    _same(dw, d[0].T @ d[2], tol)
    off = torch.tensor([0, 5, 5, rows], dtype=torch.int32, device="cuda")
    we = torch.stack([w, w, w.flip(1)])
    _same(muon.expert_linear(x, off, we), torch.cat([d[0][:5] @ d[1], d[0][5:] @ d[1].flip(1)]), tol)
    dx, dw, _ = muon.expert_linear_backward(dy, x, off, we)
    _same(dx, torch.cat([d[2][:5] @ d[1].T, d[2][5:] @ d[1].flip(1).T]), tol)
    _same(dw, torch.stack([d[0][:5].T @ d[2][:5], 0 * w.nan_to_num(0, 0, 0).double().cpu(), d[0][5:].T @ d[2][5:]]), tol)
    muon.check_ops_error()


def test_a_sum_of_more_rows_than_a_short_wait_allows():
    """150 million fp32 rows through one expert: its sum takes longer than the
    bound of the other waits (2^32 cycles).  Sums of +-1 are exact."""
    rows = 150_000_001
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GiB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randint(0, 2, (rows, 1), generator=g, device="cuda", dtype=torch.int8).float().mul_(2).sub_(1)
             for _ in range(2))
    off = torch.tensor([0, rows - 5], dtype=torch.int32, device="cuda")
    w = torch.ones(1, 1, 1, device="cuda")
    _, dw, _ = muon.expert_linear_backward(dy, x, off, w, dx=False)
    muon.check_ops_error()
    assert dw.item() == (x * dy)[:rows - 5].double().sum().item()


@pytest.mark.parametrize("rows", [3, 70])
@pytest.mark.parametrize("n_in,n_out", [((1 << 22) + 72, 8), (16, (1 << 22) + 72)])
def test_widths_past_4_million(n_in, n_out, rows):
    """Sums of +-1: exact in fp32, one rounding at the store."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w, dy = (torch.randint(0, 2, s, generator=g, device="cuda", dtype=torch.int8).bfloat16().mul_(2).sub_(1)
                for s in ((rows, n_in), (n_in, n_out), (rows, n_out)))
    d = [t.double() for t in (x, w, dy)]
    assert torch.equal(muon.linear(x, w), (d[0] @ d[1]).bfloat16())
    dx, dw, db = muon.linear_backward(dy, x, w, bias=True)
    assert torch.equal(dx, (d[2] @ d[1].T).bfloat16())
    assert torch.equal(dw, (d[0].T @ d[2]).bfloat16())
    assert torch.equal(db, d[2].sum(0).bfloat16())
    muon.check_ops_error()
