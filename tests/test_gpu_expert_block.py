"""The layer norm, the balance loss and the 4-bit products run together with the
operators they stand beside (examples/expert_layer.py): a block's result, its
gradients and its packed form against the same chain of fp64 oracle functions, in a
captured graph too."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
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


def _block(example, dtype=torch.float32):
    block = example.ExpertBlock(96, 130, 8, 3, balance=0.5, dtype=dtype, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    block.w_norm += 0.2 * torch.randn(96, generator=g, device="cuda")
    block.b_norm += 0.2 * torch.randn(96, generator=g, device="cuda")
    x, dy = (torch.randn(150, 96, generator=g, device="cuda").to(dtype) for _ in range(2))
    return block, x, dy


def _chain(x, wn, bn, wg, wu, wd, top_k, coef, dy):
    n, mean, rstd = ref.layer_norm(x, wn, bn)
    logits = n @ wg
    idx, wts = ref.gate(logits, top_k)
    xs, slot, off = ref.dispatch(n, idx, wg.shape[1])
    h, z = ref.expert_linear(xs, off, wu, kind="silu")
    ys, _ = ref.expert_linear(h, off, wd)
    y = ref.combine(ys, slot, wts, x)
    loss, counts, live = ref.balance_loss(logits, idx, coef)
    dys, dwts = ref.combine_backward(dy, ys, slot, wts)
    dh, dwd, _, _ = ref.expert_linear_backward(dys, h, off, wd)
    dxs, dwu, _, _ = ref.expert_linear_backward(dh, xs, off, wu, z, "silu")
    dlogits = ref.balance_loss_backward(1.0, logits, counts, live, coef, ref.gate_backward(dwts, logits, idx))
    dng, dwg, _, _ = ref.linear_backward(dlogits, n, wg)
    dx, dwn, dbn = ref.layer_norm_backward(ref.combine(dxs, slot) + dng, x, mean, rstd, wn, dy)
    return y, idx, loss, counts, dx, [dwg, dwu, dwd], dwn, dbn


def test_block_matches_the_oracle_chain(example):
    """fp32 throughout: each operator is within 2^-20 of its sum of magnitudes, which
    cancellation in sums of up to 130 terms raises to about 1e-4 of the result's norm at
    most."""
    block, x, dy = _block(example)
    y, saved = block.forward(x)
    dx, grads, dwn, dbn = block.backward(dy, saved)
    Y, IDX, LOSS, COUNTS, DX, G, DWN, DBN = _chain(
        to64(x), to64(block.w_norm), to64(block.b_norm), *(to64(p) for p in block.params()), 3, 0.5, to64(dy))
    assert np.array_equal(saved[3][2].cpu().numpy(), IDX) and np.array_equal(saved[5].cpu().numpy(), COUNTS)
    assert abs(float(saved[4]) - LOSS) <= 1e-5 * LOSS
    for got, want in ((y, Y), (dx, DX), (dwn, DWN), (dbn, DBN), *zip(grads, G)):
        assert np.linalg.norm(to64(got) - want) <= 1e-4 * np.linalg.norm(want)


def test_packed_block_matches_the_oracle_chain(example):
    """The tokens are rounded to 4 bits before each product: a row of h that lies
    within the fp32 error of a border may go to the other side, half a step of one
    number of 130 (6 against 4 at most).  Of 450 rows with 130 numbers each, about 450 *
    130 * 2^-18 = 0.2 do, each worth 2 / (2 sqrt 130) of a row."""
    block, x, _ = _block(example)
    block.pack()
    got = block.serve(x)
    muon.check_ops_error()
    X = to64(x)
    n, _, _ = ref.layer_norm(X, to64(block.w_norm), to64(block.b_norm))
    idx, wts = ref.gate(n @ to64(block.w_gate), 3)
    # (the rows that the products round are the GPU's own: the norm's result in fp32)
    n = to64(muon.layer_norm(x, block.w_norm, bias=block.b_norm))
    xs, slot, off = ref.dispatch(n, idx, 8)
    up, down = (np.swapaxes(ref.mx_round(np.swapaxes(to64(w), 1, 2))[0], 1, 2) for w in (block.w_up, block.w_down))
    h, _ = ref.expert_linear(ref.mx_round(xs)[0], off, up, kind="silu")
    ys, _ = ref.expert_linear(ref.mx_round(h)[0], off, down)
    want = ref.combine(ys, slot, wts, X)
    row = np.linalg.norm(to64(got) - want, axis=1) / np.linalg.norm(want, axis=1)
    assert np.median(row) <= 1e-5 and row.max() <= 0.1 and (row > 1e-4).sum() <= 8


def test_block_in_a_captured_graph(example):
    """The whole block forward, back and packed, replayed on new tokens."""
    block, x, dy = _block(example, torch.bfloat16)
    block.pack()

    def run():
        y, saved = block.forward(x)
        dx, grads, dwn, dbn = block.backward(dy, saved)
        return [y, saved[4], saved[5], dx, *grads, dwn, dbn, block.serve(x)]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    g = torch.Generator(device="cuda").manual_seed(7)
    for i in range(6):
        x.copy_(torch.randn(150, 96, generator=g, device="cuda"))
        graph.replay()
        fresh = run()
        assert all(torch.equal(p, q) for p, q in zip(held, fresh)), i
    muon.check_ops_error()


def test_the_example_runs(example):
    losses, busiest, error = example.train_block(hidden=256, inner=128, experts=8, top_k=2, tokens=512, steps=4)
    assert all(np.isfinite(losses)) and all(1 / 8 <= b <= 1 for b in busiest) and np.isfinite(error)
