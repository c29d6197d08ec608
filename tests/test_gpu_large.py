"""Tensors of more than 2^31 elements: element offsets do not fit in 32 bits.
Rows at the start, the middle and the end are checked."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

from layers_tol import U, acc

pytestmark = pytest.mark.gpu


def _need(gib):
    if torch.cuda.mem_get_info()[0] < gib * (1 << 30):
        pytest.skip(f"needs {gib} GiB of device memory")


def test_linear_output_past_32_bits():
    _need(24)
    rows, n_in, n_out = 70001, 72, 40008
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, n_in, generator=g, device="cuda").bfloat16()
    w = torch.randn(n_in, n_out, generator=g, device="cuda").bfloat16()
    y = muon.linear(x, w, activation="relu")
    muon.check_ops_error()
    pick = torch.tensor([0, 1, 26843, 53687, 53688, rows - 2, rows - 1], device="cuda")
    want = (x[pick].double() @ w.double()).clamp(min=0)
    tol = acc(n_in) * (x[pick].abs().double() @ w.abs().double()) + U[torch.bfloat16] * 1.01 * want + 1e-37
    assert ((y[pick].double() - want).abs() <= tol).all()
    del y
    # the way back: a gradient and a pre-activation of that size
    dy = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    dy[pick] = 0.5
    dx, dw, db = muon.linear_backward(dy, x, w, bias=True)
    muon.check_ops_error()
    assert torch.equal(db, torch.full_like(db, 0.5 * len(pick)))
    want = 0.5 * x[pick].double().sum(0)
    assert ((dw.double() - want[:, None]).abs() <= 2.0 ** -8 * want.abs()[:, None] + 1e-5).all()
    want = 0.5 * w.double().sum(1)
    tol = acc(n_out) * 0.5 * w.abs().double().sum(1) + 2.0 ** -8 * want.abs()
    assert ((dx[pick].double() - want).abs() <= tol).all()
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    live[pick] = True
    assert not dx[~live].any()


def test_sort_past_32_bits():
    _need(32)
    tokens, top_k, experts, hidden = 40000, 8, 64, 7168
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    idx = torch.rand(tokens, experts, generator=g, device="cuda").argsort(1)[:, :top_k].int().contiguous()
    wts = torch.full((tokens, top_k), 0.125, device="cuda")
    xs, slot, offsets = muon.dispatch(x, idx, experts)
    assert int(offsets[-1]) == tokens * top_k and xs.numel() > 1 << 31
    pick = torch.tensor([0, 7, 19999, tokens - 1], device="cuda")
    for j in range(top_k):
        assert torch.equal(xs[slot[pick, j].long()], x[pick])
    last = int(offsets[-1]) - 1  # the last row belongs to the last expert's last token
    t = int((idx == experts - 1).any(1).nonzero()[-1])
    assert torch.equal(xs[last], x[t])
    assert torch.equal(muon.combine(xs, slot, wts), x)  # eight eighths, exact in fp32
    assert torch.equal(muon.dispatch_backward(xs, slot)[pick], (8 * x[pick].float()).bfloat16())
