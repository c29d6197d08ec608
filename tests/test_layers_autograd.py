"""The layer operators build no autograd graph, and say so instead of dropping a
gradient that autograd would expect."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon


def _calls(x, w):
    i = torch.zeros(4, 2, dtype=torch.int32, device=x.device)
    off = torch.tensor([0, 4], dtype=torch.int32, device=x.device)
    f = torch.zeros(4, 2, device=x.device)
    rows = torch.zeros(8, x.shape[1], device=x.device)
    return [lambda: muon.linear(x, w), lambda: muon.linear(x.detach(), w=w), lambda: muon.linear(x, w.detach(), stream=0),
            lambda: muon.linear_backward(x, x, w), lambda: muon.expert_linear(x, off, w[None]),
            lambda: muon.expert_linear_backward(x, x, off, w[None]), lambda: muon.gate(x, 2),
            lambda: muon.gate_backward(f, x, i), lambda: muon.dispatch(x, i, 3),
            lambda: muon.dispatch_backward(rows + w[0], i),
            lambda: muon.combine(rows, i, f + w.sum()), lambda: muon.combine_backward(x, rows, i, off, f)]


def test_tensors_that_require_grad_are_refused():
    """Before anything else is looked at: these tensors are not even on a GPU."""
    x, w = torch.zeros(4, 4, requires_grad=True), torch.zeros(4, 4, requires_grad=True)
    for i, f in enumerate(_calls(x, w)):
        with pytest.raises(ValueError, match="requires grad"):
            f()
        with torch.no_grad(), pytest.raises(ValueError) as e:  # refused for where they are
            f()
        assert "requires grad" not in str(e.value), i


@pytest.mark.gpu
def test_calls_inside_an_autograd_function():
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, z = muon.linear(x, w, bias=b, activation="silu", keep_preact=True)
            ctx.save_for_backward(x, w, z)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, z = ctx.saved_tensors
            return muon.linear_backward(dy.contiguous(), x, w, preact=z, activation="silu", bias=True)

    g = torch.Generator(device="cuda").manual_seed(1)
    x, w, b = (torch.randn(*s, generator=g, device="cuda").requires_grad_() for s in ((40, 24), (24, 72), (72,)))
    with pytest.raises(ValueError, match="w requires grad"):
        muon.linear(x.detach(), w)
    dy = torch.randn(40, 72, generator=g, device="cuda")
    got = torch.autograd.grad(Linear.apply(x, w, b), (x, w, b), dy)
    d = [t.detach().double().requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad(torch.nn.functional.silu(d[0] @ d[1] + d[2]), d, dy.double())
    for p, q in zip(got, want):  # sums of up to 72 terms of size about 10, fp32
        assert (p.double() - q).abs().max() <= 72 * 10 * 2.0 ** -20
