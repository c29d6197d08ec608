"""The layer operators and the Muon update run together (examples/expert_layer.py):
the layer's result and gradients against the same chain of fp64 oracle
functions, and a training run whose loss falls."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import layers_ref as ref

from layers_tol import to64

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _chain(x, wg, wu, wd, top_k, dy):
    logits = x @ wg
    idx, wts = ref.gate(logits, top_k)
    xs, slot, off = ref.dispatch(x, idx, wg.shape[1])
    h, z = ref.expert_linear(xs, off, wu, kind="silu")
    ys, _ = ref.expert_linear(h, off, wd)
    y = ref.combine(ys, slot, wts, x)
    dys, dwts = ref.combine_backward(dy, ys, slot, wts)
    dh, dwd, _, _ = ref.expert_linear_backward(dys, h, off, wd)
    dxs, dwu, _, _ = ref.expert_linear_backward(dh, xs, off, wu, z, "silu")
    dlogits = ref.gate_backward(dwts, logits, idx)
    dxg, dwg, _, _ = ref.linear_backward(dlogits, x, wg)
    return y, idx, dy + ref.combine(dxs, slot) + dxg, [dwg, dwu, dwd]


def test_layer_matches_the_oracle_chain(example):
    """fp32 throughout: each of the nine operators is within 2^-20 of its sum of
    magnitudes, which cancellation in sums of up to 130 terms raises to about
    1e-4 of the result's norm at most."""
    layer = example.ExpertLayer(96, 130, 8, 3, dtype=torch.float32, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(150, 96, generator=g, device="cuda") for _ in range(2))
    y, saved = layer.forward(x)
    dx, grads = layer.backward(dy, saved)
    Y, IDX, DX, G = _chain(to64(x), *(to64(p) for p in layer.params()), 3, to64(dy))
    assert np.array_equal(saved[2].cpu().numpy(), IDX)
    for got, want in ((y, Y), (dx, DX), *zip(grads, G)):
        assert np.linalg.norm(to64(got) - want) <= 1e-4 * np.linalg.norm(want)


def test_training_lowers_the_loss(example):
    losses = example.train(hidden=256, inner=128, experts=8, top_k=2, tokens=512, steps=30)
    assert all(np.isfinite(losses)) and np.mean(losses[-3:]) < 0.7 * np.mean(losses[:3])
