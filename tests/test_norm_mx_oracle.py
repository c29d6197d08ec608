"""The fp64 forms of the layer norm, the balance loss and microscaled 4-bit numbers
on the host: gradients against central differences, rounding against a search over
every number there is."""
import math

import numpy as np
import pytest

from oracle import layers_ref as ref

H = 1e-5
TOL = 1e-7  # truncation h^2 f''' / 6 ~ 1e-10, rounding 1e-16 / h ~ 1e-11, sums of up to ~50 terms


def _numeric(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + H
        hi = f()
        x[i] = keep - H
        g[i] = (hi - f()) / (2 * H)
        x[i] = keep
    return g


def test_layer_norm_gradient_matches_differences():
    rng = np.random.default_rng(1)
    x, w, b, dy = rng.normal(size=(5, 7)) * 2 + 1, rng.normal(size=7), rng.normal(size=7), rng.normal(size=(5, 7))
    f = lambda: float((ref.layer_norm(x, w, b)[0] * dy).sum())  # noqa: E731
    _, mean, rstd = ref.layer_norm(x, w, b)
    dx, dw, db = ref.layer_norm_backward(dy, x, mean, rstd, w)
    for got, arr in ((dx, x), (dw, w), (db, b)):
        assert np.max(np.abs(got - _numeric(f, arr))) < TOL
    plain = ref.layer_norm(x, eps=0.0)[0]
    assert np.allclose(plain.mean(axis=1), 0) and np.allclose((plain ** 2).mean(axis=1), 1)


def test_balance_loss_gradient_matches_differences():
    rng = np.random.default_rng(2)
    logits = rng.normal(size=(6, 5))
    idx = np.array([[0, 1], [1, -1], [4, 2], [0, 9], [3, 0], [1, 2]])
    _, counts, live = ref.balance_loss(logits, idx, 0.3)
    assert counts.tolist() == [3, 3, 2, 1, 1] and live == 6
    got = ref.balance_loss_backward(1.7, logits, counts, live, 0.3)
    assert np.max(np.abs(got - _numeric(lambda: 1.7 * ref.balance_loss(logits, idx, 0.3)[0], logits))) < TOL


def test_balance_loss_of_an_even_router_and_of_padding():
    assert ref.balance_loss(np.zeros((8, 4)), np.arange(8).reshape(8, 1) % 4, 0.5)[0] == pytest.approx(0.5)
    logits = np.zeros((8, 4))
    logits[5:] = -math.inf
    loss, counts, live = ref.balance_loss(logits, np.full((8, 1), -1), 1.0)
    assert (loss, counts.sum(), live) == (0.0, 0, 5)
    assert not ref.balance_loss_backward(1.0, logits, counts, live).any()


def test_rounding_is_to_the_nearest_number_of_the_scale():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(20, 70)) * 10.0 ** rng.uniform(-30, 30, size=(20, 1))
    q, s = ref.mx_round(x)
    assert s.shape == (20, 3)
    for i in range(20):
        for b in range(3):
            part = slice(32 * b, min(32 * b + 32, 70))
            scale = 2.0 ** (int(s[i, b]) - 127)
            top = np.abs(x[i, part]).max()
            assert 4 <= top / scale < 8
            every = np.concatenate((ref.MX_GRID, -ref.MX_GRID)) * scale
            assert np.isin(q[i, part], every).all()
            err = np.abs(q[i, part] - x[i, part])
            assert (err <= np.abs(every[None] - x[i, part, None]).min(axis=1)).all()
    assert np.array_equal(ref.mx_round(q)[0], q)  # what is held comes back


def test_ties_go_to_the_even_code_and_bytes_stand_for_it():
    x = np.zeros((1, 32))
    x[0, :10] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.75, 7.9]
    q, s = ref.mx_round(x)
    assert s.tolist() == [[127]]
    assert q[0, :10].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, -1, 6]
    values = np.zeros((1, 16), dtype=np.uint8)
    values[0, 0], values[0, 4] = 0x06, 0x7a  # first in the low half: 4, 0 and -1, 6
    held = ref.mx_held(values, s, 32)
    assert held[0, :2].tolist() == [4, 0] and held[0, 8:10].tolist() == [-1, 6]


def test_the_ends_of_the_scales():
    x = np.zeros((4, 32))
    x[0, 0], x[1, 0], x[2, 3], x[3, 1] = 2.0 ** -140, 1.5 * 2.0 ** 127, math.inf, math.nan
    q, s = ref.mx_round(x)
    assert s[:, 0].tolist() == [0, 252, 255, 255]
    assert q[0, 0] == 0 and q[1, 0] == 1.5 * 2.0 ** 127 and np.isnan(q[2:]).all()
