"""The fp64 layer oracle on the host: gradients against central differences,
activations against their slopes, the sort and the gate against small
hand-written cases and invariants."""
import math

import numpy as np
import pytest

from oracle import layers_ref as ref

H = 1e-5


def _numeric(f, x):
    """Gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + H
        hi = f()
        x[i] = keep - H
        g[i] = (hi - f()) / (2 * H)
        x[i] = keep
    return g


# central differences: truncation h^2 f''' / 6 ~ 1e-10, rounding 1e-16 / h ~ 1e-11, sums of up to ~50 terms
TOL = 1e-7


@pytest.mark.parametrize("kind", ref.ACTIVATIONS)
def test_slopes_match_differences(kind):
    z = np.array([-9.0, -2.5, -0.3, 0.1, 0.7, 3.0, 11.0])
    num = (ref.act(z + H, kind) - ref.act(z - H, kind)) / (2 * H)
    assert np.max(np.abs(num - ref.act_slope(z, kind))) < TOL


@pytest.mark.parametrize("kind", ref.ACTIVATIONS)
def test_expert_linear_gradient_matches_differences(kind):
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(size=(6, 3)), rng.normal(size=(3, 3, 4)), rng.normal(size=(3, 4))
    dy = rng.normal(size=(6, 4))
    offsets = [0, 2, 2, 5]  # an empty expert and a row of none

    def f():
        return float((ref.expert_linear(x, offsets, w, b, kind)[0] * dy).sum())

    z = ref.expert_linear(x, offsets, w, b, kind)[1]
    dx, dw, db, _ = ref.expert_linear_backward(dy, x, offsets, w, z, kind)
    for got, arr in ((dx, x), (dw, w), (db, b)):
        assert np.max(np.abs(got - _numeric(f, arr))) < TOL
    assert not dx[5].any() and not dw[1].any()


@pytest.mark.parametrize("renormalize", [False, True])
def test_gate_gradient_matches_differences(renormalize):
    rng = np.random.default_rng(2)
    logits = rng.normal(size=(5, 7))
    logits[1, 2:] = -math.inf
    logits[2] = -math.inf
    g = rng.normal(size=(5, 3))
    idx, _ = ref.gate(logits, 3, renormalize)

    def f():
        wts = ref.gate(logits, 3, renormalize)[1]
        return float((wts * g).sum())

    with np.errstate(invalid="ignore"):
        num = np.where(np.isinf(logits), 0.0, _numeric(f, logits))
    assert np.max(np.abs(num - ref.gate_backward(g, logits, idx, renormalize))) < TOL


def test_gate_orders_and_masks():
    logits = np.array([[1.0, 3.0, 3.0, -math.inf], [-math.inf] * 4, [0.0, -math.inf, -math.inf, -math.inf]])
    idx, wts = ref.gate(logits, 3)
    assert idx.tolist() == [[1, 2, 0], [-1, -1, -1], [0, -1, -1]]
    assert wts[0, 0] == wts[0, 1] and abs(wts[0].sum() - 1) < 1e-15
    assert not wts[1].any() and wts[2].tolist() == [1.0, 0.0, 0.0]


def test_sort_and_back():
    x = np.arange(8.0).reshape(4, 2)
    idx = np.array([[1, 0], [1, -1], [0, 5], [2, 1]])
    xs, slot, offsets = ref.dispatch(x, idx, 4)
    assert offsets.tolist() == [0, 2, 5, 6, 6]
    assert slot.tolist() == [[2, 0], [3, -1], [1, -1], [5, 4]]
    assert np.array_equal(xs[:6], x[[0, 2, 0, 1, 3, 3]]) and not xs[6:].any()
    rng = np.random.default_rng(3)
    ys, dy, wts = rng.normal(size=(8, 2)), rng.normal(size=(4, 2)), rng.normal(size=(4, 2))
    dys, dwts = ref.combine_backward(dy, ys, slot, wts)

    def f():
        return float((ref.combine(ys, slot, wts) * dy).sum())

    assert np.max(np.abs(dys - _numeric(f, ys))) < TOL
    assert np.max(np.abs(dwts - _numeric(f, wts))) < TOL
    d = rng.normal(size=(8, 2))
    assert np.allclose((xs * d).sum(), (x * ref.combine(d, slot)).sum())  # the gather's adjoint
