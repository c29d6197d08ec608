"""The balance loss and its gradient on the GPU against the fp64 oracle: counts
exactly, the loss and its gradient within their bounds.

A probability is within rel of itself (the exponential within 4 ulp of an argument
rounded once, 2^-23 for each unit of the logits' spread; the sum over the experts).
All terms of the loss are positive, and no sum adds more than 64 + 300 of them one
after another."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import TINY, U, acc, close, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check(logits, idx, coef=1.0, residual=None):
    loss, counts, live = muon.balance_loss(logits, idx, coef=coef)
    L = to64(logits)
    LOSS, COUNTS, LIVE = ref.balance_loss(L, idx.cpu().numpy(), coef)
    assert np.array_equal(counts.cpu().numpy(), COUNTS) and int(live) == LIVE
    finite = np.where(np.isfinite(L), L, 0)
    spread = np.minimum((finite.max(1) - finite.min(1))[:, None], 110)
    rel = acc(logits.shape[1]) + (16 + 2 * spread) * 2.0 ** -23
    assert abs(float(loss) - LOSS) <= (float(rel.max()) + acc(400)) * abs(LOSS) + 1e-37
    dloss = torch.tensor(1.3, device="cuda")
    d = muon.balance_loss_backward(dloss, logits, counts, live, coef=coef, residual=residual)
    RES = None if residual is None else to64(residual)
    D = ref.balance_loss_backward(float(dloss), L, COUNTS, LIVE, coef, RES)
    open_ = np.isfinite(L)
    m = np.where(open_, L, -1e300)
    p = np.where(open_, np.exp(m - m.max(1, keepdims=True)), 0)
    p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    share = COUNTS / max(int(COUNTS.sum()), 1)
    size = abs(float(dloss) * coef) * L.shape[1] / max(LIVE, 1) * p * (share + (p * share).sum(1, keepdims=True))
    t = 4 * rel * size + (0 if residual is None else 2.0 ** -24 * np.abs(RES))
    dt = logits.dtype
    close(d, D, t + U[dt] * (np.abs(D) + t) * 1.01 + TINY[dt], "dlogits")
    return loss, counts, live


CASES = [(1, 1, 1), (1, 64, 8), (5, 2, 2), (9, 8, 4), (33, 31, 32), (100, 33, 7), (257, 64, 8), (64, 65, 1), (50, 128, 6),
         (21, 200, 8), (40, 256, 8), (17, 257, 16), (30, 512, 9), (9, 600, 9), (7, 1024, 32), (3, 1000, 2), (5000, 16, 2),
         (4096, 256, 4), (4097, 256, 4), (70000, 16, 2), (2000, 600, 3)]  # one cluster's, and just above


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_balance_loss(case, dtype):
    tokens, experts, top_k = case
    top_k = min(top_k, experts)
    g = torch.Generator(device="cuda").manual_seed(sum(case))
    logits = (torch.randn(tokens, experts, generator=g, device="cuda") * 2).to(DT[dtype])
    idx, _ = muon.gate(logits, top_k)
    _check(logits, idx, coef=0.01)
    logits[torch.rand(tokens, experts, generator=g, device="cuda") < 0.4] = -math.inf
    logits[::5] = -math.inf
    idx, _ = muon.gate(logits, top_k)
    r = torch.randn(tokens, experts, generator=g, device="cuda").to(DT[dtype])
    _check(logits, idx, residual=r)


def test_indices_from_elsewhere():
    """The same expert twice, numbers of no expert, nothing at all."""
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(300, 24, generator=g, device="cuda")
    idx = torch.randint(-3, 30, (300, 5), generator=g, device="cuda", dtype=torch.int32)
    _check(logits, idx)
    _check(logits, torch.full_like(idx, 7))
    _check(logits, torch.full_like(idx, -1))
    idx[0, 0], idx[0, 1] = 2 ** 31 - 1, -2 ** 31
    _check(logits, idx)
    _check(torch.full_like(logits, -math.inf), idx)


def test_extreme_and_non_finite_logits():
    low = torch.finfo(torch.float32).min
    rows = torch.zeros(5, 12, device="cuda")
    rows[0] = low                    # masks by the lowest value: still open, all alike
    rows[1] = low
    rows[1, 3] = 5.0
    rows[2] = torch.arange(12) * 9.0
    rows[3] = 3e38
    rows[4] = -math.inf
    rows[4, 11] = -3e38              # the only one left
    idx, _ = muon.gate(rows, 4)
    _check(rows, idx)
    rows[2, 5] = math.nan
    loss, counts, live = muon.balance_loss(rows, idx)
    assert math.isnan(float(loss)) and int(live) == 5
    d = muon.balance_loss_backward(torch.ones((), device="cuda"), rows, counts, live)
    assert torch.isnan(d[2]).any() and torch.isfinite(d[[0, 1, 3, 4]]).all()


def test_many_tokens_keep_their_digits():
    """Even logits: every probability is 1/64 exactly, and so is the loss, whatever the
    number of tokens."""
    for tokens in (100003, 2000003):
        logits = torch.zeros(tokens, 64, dtype=torch.bfloat16, device="cuda")
        idx = (torch.arange(tokens, device="cuda", dtype=torch.int32) % 64)[:, None].contiguous()
        loss, counts, live = muon.balance_loss(logits, idx)
        assert int(live) == tokens and int(counts.sum()) == tokens
        assert abs(float(loss) - 1.0) <= acc(400)


def test_strides_streams_graphs_and_no_tokens():
    g = torch.Generator(device="cuda").manual_seed(2)
    wide = torch.randn(70, 100, generator=g, device="cuda").bfloat16()
    for cut in (slice(11, 61), slice(16, 80)):
        part, whole = wide[:, cut], wide[:, cut].contiguous()
        idx, _ = muon.gate(part, 4)
        want = muon.balance_loss(whole, idx)
        got = muon.balance_loss(part, idx)
        assert torch.equal(got[1], want[1])
        close(got[0], to64(want[0]), acc(300) * to64(want[0]), "loss")
        _check(part, idx, residual=torch.randn(70, 100, generator=g, device="cuda").bfloat16()[:, cut])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    there = muon.balance_loss(part, idx, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(there, got))
    none = muon.balance_loss(part[:0], idx[:0])
    assert float(none[0]) == 0 and not none[1].any() and int(none[2]) == 0
    assert muon.balance_loss_backward(none[0], part[:0], none[1], none[2]).shape == (0, 64)
    logits = torch.randn(500, 64, generator=g, device="cuda")
    one = torch.ones((), device="cuda")

    def run():
        idx, _ = muon.gate(logits, 8)
        out = muon.balance_loss(logits, idx)
        return (*out, muon.balance_loss_backward(one, logits, out[1], out[2]))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(5):
        logits.copy_(torch.randn(500, 64, generator=g, device="cuda"))
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(held, run())), i


def test_gradient_matches_differences():
    """Central differences of the fp32 loss along random directions (the choice is an
    input): off by h^2 f''' / 6 < 1e-4 * 30 / 6 and by 2^-21 of the loss over h."""
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(40, 24, generator=g, device="cuda")
    idx, _ = muon.gate(logits, 3)
    _, counts, live = muon.balance_loss(logits, idx)
    d = muon.balance_loss_backward(torch.ones((), device="cuda"), logits, counts, live)
    for _ in range(5):
        v = torch.randn(40, 24, generator=g, device="cuda")
        hi, lo = (float(muon.balance_loss(logits + s * 1e-2 * v, idx)[0]) for s in (1, -1))
        assert abs((hi - lo) / 2e-2 - float((d * v).sum())) < 1e-3


def test_refusals():
    x = torch.randn(4, 16, device="cuda")
    idx, _ = muon.gate(x, 3)
    loss, counts, live = muon.balance_loss(x, idx)
    for f in (lambda: muon.balance_loss(x[0], idx), lambda: muon.balance_loss(x.double(), idx),
              lambda: muon.balance_loss(x, idx.long()), lambda: muon.balance_loss(x, idx[:2]),
              lambda: muon.balance_loss(x, idx.cpu()), lambda: muon.balance_loss(x.t(), idx),
              lambda: muon.balance_loss_backward(loss.double(), x, counts, live),
              lambda: muon.balance_loss_backward(x[0], x, counts, live),
              lambda: muon.balance_loss_backward(loss, x, counts[:3], live),
              lambda: muon.balance_loss_backward(loss, x, counts, live.long()),
              lambda: muon.balance_loss_backward(loss, x, counts, live, residual=x.half())):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(muon.MuonError):
        muon.balance_loss(x, idx, coef=math.inf)
    with pytest.raises(muon.MuonError):
        muon.balance_loss(torch.randn(2, 1025, device="cuda"), idx[:2])
