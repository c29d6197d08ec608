"""Tokens into expert order and back, and the gradients, on the GPU against the
fp64 oracle: the order exactly, rows bit for bit, sums within their bounds."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import TINY, U, acc, close, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _case(tokens, top_k, experts, hidden, dtype, seed, drop=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.rand(tokens, experts, generator=g, device="cuda").argsort(1)[:, :top_k].int().contiguous()
    if drop:
        out = torch.rand(tokens, top_k, generator=g, device="cuda")
        idx[out < drop] = -1
        idx[out < drop / 2] = experts + 3
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    wts = torch.rand(tokens, top_k, generator=g, device="cuda")
    return idx, wts, n(tokens, hidden), n(tokens * top_k, hidden), n(tokens, hidden), n(tokens * top_k, hidden), n(tokens, hidden)


CASES = [(1, 1, 1, 1), (1, 8, 64, 7168), (3, 2, 5, 17), (7, 4, 8, 64), (33, 6, 48, 100), (130, 8, 256, 72),
         (257, 2, 1024, 33), (1000, 1, 3, 40), (700, 3, 40, 264), (2, 32, 32, 8), (1500, 8, 60, 16)]


@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_sort_and_back(case, dtype, drop):
    dt = DT[dtype]
    tokens, top_k, experts, hidden = case
    idx, wts, x, ys, r, dxs, dy = _case(*case, dt, seed=sum(case), drop=drop)
    xs, slot, offsets = muon.dispatch(x, idx, experts)
    XS, SLOT, OFF = ref.dispatch(to64(x), idx.cpu().numpy(), experts)
    assert np.array_equal(slot.cpu().numpy(), SLOT) and np.array_equal(offsets.cpu().numpy(), OFF)
    assert np.array_equal(to64(xs), XS)
    xs2, slot2, offsets2 = muon.dispatch(x, idx.long(), experts)
    assert torch.equal(xs, xs2) and torch.equal(slot, slot2) and torch.equal(offsets, offsets2)

    W, YS, R, DXS, DY = to64(wts), to64(ys), to64(r), to64(dxs), to64(dy)
    for rr, name in ((r, "residual"), (None, "plain")):
        y = muon.combine(ys, slot, wts, residual=rr)
        Y = ref.combine(YS, SLOT, W, None if rr is None else R)
        t = acc(top_k) * (ref.combine(np.abs(YS), SLOT, W) + (0 if rr is None else np.abs(R)))
        close(y, Y, t + U[dt] * (np.abs(Y) + t) * 1.01 + TINY[dt], name)
    dx = muon.dispatch_backward(dxs, slot)
    DX = ref.combine(DXS, SLOT)
    t = acc(top_k) * ref.combine(np.abs(DXS), SLOT)
    close(dx, DX, t + U[dt] * (np.abs(DX) + t) * 1.01 + TINY[dt], "dx")
    dys, dwts = muon.combine_backward(dy, ys, slot, offsets, wts)
    DYS, DW = ref.combine_backward(DY, YS, SLOT, W)
    close(dys, DYS, (U[dt] + 2.0 ** -23) * np.abs(DYS) * 1.01 + TINY[dt], "dys")
    close(dwts, DW, acc(hidden) * ref.combine_backward(np.abs(DY), np.abs(YS), SLOT, W)[1] + 1e-37, "dweights")


def test_many_assignments_keep_their_order():
    """More than 100 blocks' worth of assignments, two experts taking most."""
    g = torch.Generator(device="cuda").manual_seed(7)
    idx = torch.randint(0, 37, (30011, 4), generator=g, device="cuda", dtype=torch.int32)
    idx[torch.rand(30011, 4, generator=g, device="cuda") < 0.4] = 5
    idx[torch.rand(30011, 4, generator=g, device="cuda") < 0.1] = -1
    x = torch.arange(30011, device="cuda", dtype=torch.float32)[:, None].contiguous()
    xs, slot, offsets = muon.dispatch(x, idx, 37)
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, 37)
    order = torch.sort(key, stable=True)[1]
    n = int((flat >= 0).sum())
    assert int(offsets[-1]) == n
    assert torch.equal(xs[:n, 0].long(), order[:n] // 4) and not xs[n:].any()
    s = slot.reshape(-1)
    assert torch.equal(s[order[:n]].long(), torch.arange(n, device="cuda")) and (s[flat < 0] == -1).all()
    assert torch.equal(offsets.long(), torch.searchsorted(key.sort()[0], torch.arange(38, device="cuda")))


@pytest.mark.parametrize("tokens,top_k,experts", [(1025, 1, 7), (513, 2, 1024), (3000, 3, 300), (8192, 8, 64),
                                                  (65536, 1, 5), (65537, 1, 1024)])
def test_order_of_any_number(tokens, top_k, experts):
    """One block, one cluster of blocks, many blocks: the stable sort by expert."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    idx = torch.randint(0, experts, (tokens, top_k), generator=g, device="cuda", dtype=torch.int32)
    idx[torch.rand(tokens, top_k, generator=g, device="cuda") < 0.3] = experts // 2
    idx[torch.rand(tokens, top_k, generator=g, device="cuda") < 0.1] = -1
    x = torch.arange(tokens, device="cuda", dtype=torch.float32)[:, None].contiguous()
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, experts)
    order = torch.sort(key, stable=True)[1]
    n = int((flat >= 0).sum())
    for _ in range(2):
        xs, slot, offsets = muon.dispatch(x, idx, experts)
        s = slot.reshape(-1)
        assert torch.equal(s[order[:n]].long(), torch.arange(n, device="cuda")) and (s[flat < 0] == -1).all()
        assert torch.equal(xs[:n, 0].long(), order[:n] // top_k) and not xs[n:].any()
        assert torch.equal(offsets.long(), torch.searchsorted(key.sort()[0], torch.arange(experts + 1, device="cuda")))


def test_all_to_one_and_all_dropped():
    x = torch.randn(300, 24, device="cuda").bfloat16()
    one = torch.full((300, 1), 6, dtype=torch.int32, device="cuda")
    xs, slot, offsets = muon.dispatch(x, one, 9)
    assert torch.equal(xs, x) and offsets.tolist() == [0] * 7 + [300] * 3
    none = torch.full((300, 2), -1, dtype=torch.int32, device="cuda")
    xs, slot, offsets = muon.dispatch(x, none, 9)
    assert not xs.any() and (slot == -1).all() and not offsets.any()
    wts = torch.ones(300, 2, device="cuda")
    bad = torch.full((600, 24), math.nan, device="cuda").bfloat16()
    assert not muon.combine(bad, slot, wts).any()
    assert torch.equal(muon.combine(bad, slot, wts, residual=x), x)
    dys, dw = muon.combine_backward(x, bad, slot, offsets, wts)
    assert not dys.any() and not dw.any() and not muon.dispatch_backward(bad, slot).any()


def test_non_finite_rows_stay_in_their_token():
    idx = torch.tensor([[0, 1], [1, 2], [0, 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 40, device="cuda").half()
    x[1] = math.nan
    xs, slot, offsets = muon.dispatch(x, idx, 3)
    wts = torch.full((3, 2), 0.5, device="cuda")
    y = muon.combine(xs, slot, wts)
    assert torch.equal(y[[0, 2]], x[[0, 2]]) and torch.isnan(y[1]).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_no_tokens(dtype):
    dt = DT[dtype]
    idx, wts, x, ys, r, dxs, dy = _case(50, 3, 7, 96, dt, 21, drop=0.1)
    wide = lambda t: torch.cat([t, t], 1)[:, 5:101] * 1  # noqa: E731
    sl = lambda t: torch.nn.functional.pad(t, (3, 6))[:, 3:99]  # noqa: E731
    xs, slot, offsets = muon.dispatch(x, idx, 7)
    xs2, slot2, _ = muon.dispatch(sl(x), idx, 7)
    assert torch.equal(xs, xs2) and torch.equal(slot, slot2) and not sl(x).is_contiguous() and wide(x).is_contiguous()
    assert torch.equal(muon.combine(sl(ys), slot, wts, residual=sl(r)), muon.combine(ys, slot, wts, residual=r))
    assert torch.equal(muon.dispatch_backward(sl(dxs), slot), muon.dispatch_backward(dxs, slot))
    a, b = (muon.combine_backward(f(dy), f(ys), slot, offsets, wts) for f in (sl, lambda t: t))
    assert torch.equal(a[0], b[0]) and torch.allclose(a[1], b[1], rtol=0, atol=96 * 2.0 ** -23 * 96)
    e = torch.empty(0, 96, dtype=dt, device="cuda")
    xs, slot, offsets = muon.dispatch(e, idx[:0], 7)
    assert xs.shape == (0, 96) and slot.shape == (0, 3) and not offsets.any()
    assert muon.combine(e, slot, wts[:0]).shape == (0, 96) and muon.dispatch_backward(e, slot).shape == (0, 96)
    assert muon.combine_backward(e, e, slot, offsets, wts[:0])[1].shape == (0, 3)


def test_gradient_is_the_adjoint():
    """<combine(ys, w), dy> is linear in ys and in w: its gradients give the
    same number back, up to the fp32 rounding of 200 x 64 products."""
    idx, wts, x, ys, r, dxs, dy = _case(200, 4, 16, 64, torch.float32, 22, drop=0.1)
    xs, slot, offsets = muon.dispatch(x, idx, 16)
    whole = (muon.combine(ys, slot, wts).double() * dy.double()).sum().item()
    dys, dw = muon.combine_backward(dy, ys, slot, offsets, wts)
    size = (wts.double() * 1).sum().item() * 64
    tol = size * 3 * 2.0 ** -20
    assert abs((dys.double() * ys.double()).sum().item() - whole) < tol
    assert abs((dw.double() * wts.double()).sum().item() - whole) < tol
    moved = (xs.double() * dxs.double()).sum().item()
    assert abs((x.double() * muon.dispatch_backward(dxs, slot).double()).sum().item() - moved) < 200 * 4 * 64 * 2.0 ** -20


def test_streams_graphs_and_repeats():
    idx, wts, x, ys, r, dxs, dy = _case(600, 8, 64, 256, torch.bfloat16, 23)
    xs, slot, offsets = muon.dispatch(x, idx, 64)
    want = (xs, slot, offsets, muon.combine(ys, slot, wts, residual=r), muon.dispatch_backward(dxs, slot),
            *muon.combine_backward(dy, ys, slot, offsets, wts))

    def go(**kw):
        a, b, c = muon.dispatch(x, idx, 64, **kw)
        return (a, b, c, muon.combine(ys, b, wts, residual=r, **kw), muon.dispatch_backward(dxs, b, **kw),
                *muon.combine_backward(dy, ys, b, c, wts, **kw))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = go(stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(side, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = go()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_refusals():
    idx, wts, x, ys, r, dxs, dy = _case(6, 2, 4, 16, torch.float32, 24)
    xs, slot, offsets = muon.dispatch(x, idx, 4)
    bad = [lambda: muon.dispatch(x, idx.short(), 4), lambda: muon.dispatch(x, idx[:3], 4),
           lambda: muon.dispatch(x[0], idx, 4), lambda: muon.dispatch(x.cpu(), idx, 4),
           lambda: muon.dispatch(x, idx.t().contiguous().t(), 4), lambda: muon.combine(ys[:5], slot, wts),
           lambda: muon.combine(ys, slot, wts.half()), lambda: muon.combine(ys, slot, wts, residual=r.half()),
           lambda: muon.combine(ys, slot.long(), wts), lambda: muon.dispatch_backward(dxs[:4], slot),
           lambda: muon.combine_backward(dy[:2], ys, slot, offsets, wts),
           lambda: muon.combine_backward(dy, ys, slot, offsets[:1], wts)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for experts in (0, 1025):
        with pytest.raises(muon.MuonError):
            muon.dispatch(x, idx, experts)
    with pytest.raises(muon.MuonError):
        muon.dispatch(x, torch.zeros(6, 33, dtype=torch.int32, device="cuda"), 4)
