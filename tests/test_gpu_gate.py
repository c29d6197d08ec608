"""The gate and its gradient on the GPU against the fp64 oracle: the choice
exactly, weights within their bounds; ties, masks, non-finite logits."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import TINY, U, acc, close, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check(logits, top_k, renormalize, seed=0):
    idx, wts = muon.gate(logits, top_k, renormalize=renormalize)
    IDX, WTS = ref.gate(to64(logits), top_k, renormalize)
    assert np.array_equal(idx.cpu().numpy(), IDX)
    # each term: exponential within 4 ulp of an argument rounded once (2^-24 |difference|, 2^-23 per unit of it)
    L = to64(logits)
    finite = np.where(np.isfinite(L), L, 0)
    spread = np.minimum((finite.max(1) - finite.min(1))[:, None], 110)
    rel = acc(logits.shape[1]) + (16 + 2 * spread) * 2.0 ** -23
    assert np.array_equal(np.isnan(to64(wts)), np.isnan(WTS))
    close(torch.nan_to_num(wts), np.nan_to_num(WTS), rel * np.nan_to_num(WTS) + 1e-37, "weights")
    if np.isnan(WTS).any():
        return
    g = torch.randn(wts.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    d = muon.gate_backward(g, logits, idx, renormalize=renormalize)
    D = ref.gate_backward(to64(g), to64(logits), IDX, renormalize)
    dt = logits.dtype
    p = np.zeros(L.shape)
    if renormalize:
        for t, j in zip(*np.nonzero(IDX >= 0)):
            p[t, IDX[t, j]] = 1
        over = p > 0
    else:
        over = L != -math.inf
    m = np.where(over, L, -1e300)
    p = np.where(over, np.exp(m - m.max(1, keepdims=True)), 0)
    p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    size = p * (np.abs(to64(g)).max(1, keepdims=True) * 2)
    close(d, D, 4 * rel * size + U[dt] * np.abs(D) * 1.01 + TINY[dt], "dlogits")


CASES = [(1, 1, 1), (1, 64, 8), (5, 2, 2), (9, 31, 4), (33, 32, 32), (100, 33, 7), (257, 64, 8), (64, 65, 1),
         (50, 128, 6), (21, 200, 8), (40, 256, 8), (17, 384, 16), (9, 600, 9), (7, 1024, 32), (3, 1000, 2)]


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_gate(case, dtype, renormalize):
    tokens, experts, top_k = case
    g = torch.Generator(device="cuda").manual_seed(sum(case))
    logits = (torch.randn(tokens, experts, generator=g, device="cuda") * 2).to(DT[dtype])
    _check(logits, top_k, renormalize)
    logits[torch.rand(tokens, experts, generator=g, device="cuda") < 0.4] = -math.inf
    logits[::5] = -math.inf
    _check(logits, top_k, renormalize)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts", [8, 64, 100, 512])
def test_ties_go_to_the_lower_expert(experts, renormalize):
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randint(-2, 3, (200, experts), generator=g, device="cuda").float()
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = -0.0, 0.0
    _check(logits, 8, renormalize)
    idx, _ = muon.gate(logits[:2].contiguous(), 8)
    assert idx.tolist() == [list(range(8))] * 2


def test_extreme_logits():
    low = torch.finfo(torch.float32).min
    rows = torch.zeros(6, 12, device="cuda")
    rows[0] = low                    # masks by the lowest value: still open, all alike
    rows[1] = low
    rows[1, 3] = 5.0                 # one open, the others too low to weigh anything
    rows[2] = torch.arange(12) * 30.0
    rows[3] = 3e38
    rows[4] = -math.inf
    rows[4, 11] = -3e38              # the only one left
    rows[5, 2] = 1e38
    for renormalize in (False, True):
        _check(rows, 4, renormalize)


def test_non_finite_logits():
    rows = torch.randn(4, 40, device="cuda")
    rows[1, 7] = math.nan
    rows[2] = math.nan
    idx, wts = muon.gate(rows, 5)
    IDX, _ = ref.gate(to64(rows), 5)
    assert np.array_equal(idx.cpu().numpy(), IDX)
    assert torch.isnan(wts[1]).all() and (idx[2] == -1).all() and not wts[2].any()
    assert torch.isfinite(wts[[0, 3]]).all()
    d = muon.gate_backward(torch.ones_like(wts), rows, idx, renormalize=False)
    assert torch.isfinite(d[[0, 3]]).all()


def test_strides_streams_and_no_tokens():
    wide = torch.randn(70, 100, device="cuda").bfloat16()
    part = wide[:, 11:61]
    idx, wts = muon.gate(part, 4)
    want = muon.gate(part.contiguous(), 4)
    assert torch.equal(idx, want[0]) and torch.equal(wts, want[1])
    g = torch.randn_like(wts)
    assert torch.equal(muon.gate_backward(g, part, idx), muon.gate_backward(g, part.contiguous(), idx))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i2, w2 = muon.gate(part, 4, stream=s)
    s.synchronize()
    assert torch.equal(idx, i2) and torch.equal(wts, w2)
    i0, w0 = muon.gate(part[:0], 4)
    assert i0.shape == (0, 4) and muon.gate_backward(w0, part[:0], i0).shape == (0, 50)


@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_matches_differences(renormalize):
    """Central differences of the fp32 weights along random directions that
    keep the choice: off by h^2 f''' / 6 and by 2^-23 of the sum over h."""
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(50, 24, generator=g, device="cuda") * 2
    dw = torch.randn(50, 6, generator=g, device="cuda")
    idx, _ = muon.gate(logits, 6, renormalize=renormalize)
    grad = muon.gate_backward(dw, logits, idx, renormalize=renormalize)
    d = torch.randn(50, 24, generator=g, device="cuda")
    h = 1e-2
    hi, lo = (muon.gate(logits + s * h * d, 6, renormalize=renormalize) for s in (1, -1))
    same = ((hi[0] == idx) & (lo[0] == idx)).all(1)
    assert int(same.sum()) > 25
    num = ((hi[1] - lo[1]).double() * dw.double()).sum(1) / (2 * h)
    got = (grad.double() * d.double()).sum(1)
    # third derivative of a weight along d: below 10 max|d|^3 ~ 300 for |d| ~ 3; 1e-4 * 300 / 6 = 5e-3 times |dw| ~ 3
    assert ((num - got).abs()[same] < 1.5e-2).all()


def test_refusals():
    x = torch.randn(4, 16, device="cuda")
    idx, wts = muon.gate(x, 3)
    for f in (lambda: muon.gate(x.cpu(), 3), lambda: muon.gate(x[0], 3), lambda: muon.gate(x.double(), 3),
              lambda: muon.gate(x.t(), 3), lambda: muon.gate_backward(wts.half(), x, idx),
              lambda: muon.gate_backward(wts, x, idx.long()), lambda: muon.gate_backward(wts[:2], x, idx)):
        with pytest.raises(ValueError):
            f()
    for k in (0, 17):
        with pytest.raises(muon.MuonError):
            muon.gate(x, k)
    with pytest.raises(muon.MuonError):
        muon.gate(torch.randn(2, 1025, device="cuda"), 3)
