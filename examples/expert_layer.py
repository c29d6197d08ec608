"""One training step of an expert layer with the layer operators and the Muon update.

A gate picks top_k experts for each token, the tokens are copied into expert
order, go through the experts' two matrices, come back weighted, and are added to
the layer's input.  The backward pass returns the gradients of the gate's
matrix and of both expert tensors, which one ``MuonPlan.step`` turns into an
update; every expert of [experts, in, out] is its own matrix to the plan.

    python examples/expert_layer.py [--steps N] [--tokens T]

trains the layer to imitate a fixed random one and prints the loss.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_bucket_gb300 as muon  # noqa: E402


class ExpertLayer:
    def __init__(self, hidden, inner, experts, top_k, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def matrix(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-2] ** -0.5).to(dtype)

        self.experts, self.top_k = experts, top_k
        self.w_gate = matrix(hidden, experts)
        self.w_up = matrix(experts, hidden, inner)
        self.w_down = matrix(experts, inner, hidden)

    def params(self):
        return [self.w_gate, self.w_up, self.w_down]

    def forward(self, x):
        """y = x + sum over the token's experts of weight * down(silu(up(x))), and what the way back needs."""
        logits = muon.linear(x, self.w_gate)
        idx, wts = muon.gate(logits, self.top_k)
        xs, slot, offsets = muon.dispatch(x, idx, self.experts)
        h, z = muon.expert_linear(xs, offsets, self.w_up, activation="silu", keep_preact=True)
        ys = muon.expert_linear(h, offsets, self.w_down)
        y = muon.combine(ys, slot, wts, residual=x)
        return y, (x, logits, idx, wts, xs, slot, offsets, h, z, ys)

    def backward(self, dy, saved):
        """(dx, gradients of params()) for the gradient dy of forward's result."""
        x, logits, idx, wts, xs, slot, offsets, h, z, ys = saved
        dys, dwts = muon.combine_backward(dy, ys, slot, offsets, wts)
        dh, dw_down, _ = muon.expert_linear_backward(dys, h, offsets, self.w_down)
        dxs, dw_up, _ = muon.expert_linear_backward(dh, xs, offsets, self.w_up, preact=z, activation="silu")
        dlogits = muon.gate_backward(dwts, logits, idx)
        dx_gate, dw_gate, _ = muon.linear_backward(dlogits, x, self.w_gate)
        dx = dy + muon.dispatch_backward(dxs, slot) + dx_gate
        return dx, [dw_gate, dw_up, dw_down]


def train(hidden=1024, inner=512, experts=32, top_k=4, tokens=4096, steps=20, lr=0.02, seed=0):
    """Losses of `steps` steps towards a fixed random layer of the same shape."""
    teacher = ExpertLayer(hidden, inner, experts, top_k, seed=seed + 1)
    layer = ExpertLayer(hidden, inner, experts, top_k, seed=seed + 2)
    params = layer.params()
    plan = muon.MuonPlan([list(p.shape) for p in params], scale="rms_0_2")
    momenta = [torch.zeros(p.shape, device="cuda") for p in params]
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for i in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
        target, _ = teacher.forward(x)
        y, saved = layer.forward(x)
        diff = y.float() - target.float()
        losses.append(float((diff * diff).mean()))
        _, grads = layer.backward((2.0 / diff.shape[0] * diff).bfloat16(), saved)
        plan.step(params, grads, momenta, beta=0.9, lr=lr * (1 - i / steps), wd=0.0)
    muon.check_ops_error()
    plan.check_error()
    plan.close()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    a = ap.parse_args()
    train(steps=2, tokens=a.tokens)  # warm-up: kernel attributes, the plan's graph
    t = time.perf_counter()
    losses = train(steps=a.steps, tokens=a.tokens)
    print(f"{a.steps} steps of {a.tokens} tokens in {time.perf_counter() - t:.3f} s")
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"last       loss {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
