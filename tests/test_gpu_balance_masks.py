"""The balance loss's gradient in tokens with a NaN or an infinite logit: NaN in every
open expert, those whose probability underflows beside the others included, as the
formula and the loss have it.  What masks an expert is its logit of -inf alone."""
import math

import pytest
import torch

import newton_schulz_bucket_gb300 as muon

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("experts", [3, 12, 64, 200, 264, 300, 512, 520, 777, 1024])
def test_non_finite_tokens_are_nan_in_every_open_expert(experts, dtype, residual):
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(experts)
    logits = (torch.randn(70, experts, generator=g, device="cuda") * 2).to(dt)
    # half of the experts underflow beside the others (e^-400 is 0 in 32 bits), a few are masked
    logits[:, ::2] -= 400
    logits[:, 1] = 5.0
    logits[torch.rand(70, experts, generator=g, device="cuda") < 0.2] = -math.inf
    idx = torch.randint(0, experts, (70, 2), generator=g, device="cuda", dtype=torch.int32)
    r = torch.randn(70, experts, generator=g, device="cuda").to(dt) if residual else None
    _, counts, live = muon.balance_loss(logits, idx)
    one = torch.ones((), device="cuda")
    clean = muon.balance_loss_backward(one, logits, counts, live, residual=r)
    bad = logits.clone()
    rows = {7: (0, math.nan), 20: (experts - 1, math.nan), 33: (1, math.inf), 41: (0, math.inf), 69: (2, math.nan)}
    for t, (e, v) in rows.items():
        bad[t, e] = v
    loss, _, bad_live = muon.balance_loss(bad, idx)
    assert math.isnan(float(loss)) and int(bad_live) >= int(live)
    d = muon.balance_loss_backward(one, bad, counts, live, residual=r)
    for t in range(70):
        if t not in rows:
            assert torch.equal(d[t], clean[t]), t
            continue
        masked = bad[t] == -math.inf
        want = torch.zeros(experts, dtype=dt, device="cuda") if r is None else r[t]
        assert torch.isnan(d[t][~masked]).all(), t
        assert torch.equal(d[t][masked], want[masked]), t


def test_underflowed_and_masked_experts_of_finite_tokens():
    """Both get the residual alone, and 0 without one."""
    logits = torch.zeros(4, 40, device="cuda")
    logits[:, 5:20] = -500.0
    logits[:, 30:] = -math.inf
    idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    _, counts, live = muon.balance_loss(logits, idx)
    d = muon.balance_loss_backward(torch.ones((), device="cuda"), logits, counts, live)
    assert not d[:, 5:20].any() and not d[:, 30:].any() and (d[:, 0] > 0).all() and (d[:, 1:5] < 0).all()
    r = torch.randn(4, 40, device="cuda")
    d = muon.balance_loss_backward(torch.ones((), device="cuda"), logits, counts, live, residual=r)
    assert torch.equal(d[:, 5:20], r[:, 5:20]) and torch.equal(d[:, 30:], r[:, 30:])
