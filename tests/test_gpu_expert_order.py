"""Routing followed at once by the products it feeds, in one captured graph whose
indices change from replay to replay: every kernel starts while the one before it
drains, and reads that one's offsets only when they are written."""
import random

import pytest
import torch

import newton_schulz_bucket_gb300 as muon

pytestmark = pytest.mark.gpu


# 30 and 600 tokens take the one-launch and the cluster form of the order, 9000
# the three launches; in = 129 makes the weights a padded copy
@pytest.mark.parametrize("n_in", [128, 129])
@pytest.mark.parametrize("tokens", [30, 600, 9000])
def test_products_follow_changing_offsets(tokens, n_in):
    experts, n_out, top_k = 16, 96, 2
    g = torch.Generator(device="cuda").manual_seed(tokens + n_in)
    x = torch.randn(tokens, n_in, generator=g, device="cuda").bfloat16()
    w = (torch.randn(experts, n_in, n_out, generator=g, device="cuda") / 11).bfloat16()
    idx = torch.zeros(tokens, top_k, dtype=torch.int32, device="cuda")

    pick = random.Random(n_in)

    def run():
        xs, slot, offsets = muon.dispatch(x, idx, experts)
        ys = muon.expert_linear(xs, offsets, w)
        dxs, dw, db = muon.expert_linear_backward(ys, xs, offsets, w, bias=True)
        return xs, slot, offsets, ys, dxs, dw, db

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(24):
        # a few experts at a time, others empty, some assignments dropped
        idx.copy_((pick.randrange(experts) + torch.randint(-1, 5, idx.shape, generator=g, device="cuda")) % (experts + 1) - 1)
        graph.replay()
        xs, slot, offsets, ys, dxs, dw, db = held
        want = torch.searchsorted(idx.reshape(-1).sort()[0], torch.arange(experts + 1, device="cuda", dtype=torch.int32))
        want = (want - want[0]).int()
        assert torch.equal(offsets, want), i
        off = want.tolist()
        for e in range(experts):
            rows = xs[off[e]:off[e + 1]].double()
            z = rows @ w[e].double()
            assert torch.allclose(ys[off[e]:off[e + 1]].double(), z, rtol=2.0 ** -8, atol=2e-3), (i, e)
            d = ys[off[e]:off[e + 1]].double()
            assert torch.allclose(dw[e].double(), rows.T @ d, rtol=2.0 ** -8, atol=2e-3 * max(1, len(rows)) ** 0.5), (i, e)
            assert torch.allclose(db[e].double(), d.sum(0), rtol=2.0 ** -8, atol=2e-3 * max(1, len(rows)) ** 0.5), (i, e)
        assert not ys[off[-1]:].any() and not dxs[off[-1]:].any()
    muon.check_ops_error()
