"""The layer operators in plain fp64 NumPy: a layer's product with its
epilogue, the same per expert, the gate, and tokens into expert order and
back, with the formulas of their gradients."""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


def act(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "none":
        return z
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "silu":
        return z * _sigmoid(z)
    if kind == "gelu":
        return z * _erfc(-z / math.sqrt(2.0)) / 2.0
    if kind == "gelu_tanh":
        return z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))) / 2.0
    raise KeyError(kind)


def act_slope(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = _sigmoid(z)
        return s + z * s * (1.0 - s)
    if kind == "gelu":
        return _erfc(-z / math.sqrt(2.0)) / 2.0 + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return (1.0 + t) / 2.0 + z * (1.0 - t * t) / 2.0 * c * (1.0 + 3 * 0.044715 * z * z)
    raise KeyError(kind)


def linear(x, w, b=None, kind="none", r=None):
    """(y, z)"""
    z = x @ w
    if b is not None:
        z = z + b
    y = act(z, kind)
    return (y if r is None else y + r), z


def linear_backward(dy, x, w, z=None, kind="none"):
    """(dx, dw, db, dz)"""
    dz = dy if kind == "none" else dy * act_slope(z, kind)
    return dz @ w.T, x.T @ dz, dz.sum(axis=0), dz


def expert_linear(x, offsets, w, b=None, kind="none", r=None):
    y = np.zeros((x.shape[0], w.shape[2]))
    z = np.zeros_like(y)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        y[s], z[s] = linear(x[s], w[e], None if b is None else b[e], kind, None if r is None else r[s])
    return y, z


def expert_linear_backward(dy, x, offsets, w, z=None, kind="none"):
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    db, dz = np.zeros((w.shape[0], w.shape[2])), np.zeros_like(dy)
    for e in range(w.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        dx[s], dw[e], db[e], dz[s] = linear_backward(dy[s], x[s], w[e], None if z is None else z[s], kind)
    return dx, dw, db, dz


def gate(logits, top_k, renormalize=True):
    """(indices, weights), token by token."""
    tokens, experts = logits.shape
    idx = np.full((tokens, top_k), -1, dtype=np.int32)
    wts = np.zeros((tokens, top_k))
    for t in range(tokens):
        row = [float(v) for v in logits[t]]
        nan = any(math.isnan(v) for v in row)
        open_ = [e for e in range(experts) if not math.isnan(row[e]) and row[e] != -math.inf]
        chosen = sorted(open_, key=lambda e: (-row[e], e))[:top_k]
        if not chosen:
            continue
        high = row[chosen[0]]
        over = chosen if renormalize else open_
        total = sum(math.exp(row[e] - high) for e in over)
        for j, e in enumerate(chosen):
            idx[t, j] = e
            wts[t, j] = math.nan if nan else math.exp(row[e] - high) / total
    return idx, wts


def gate_backward(dweights, logits, indices, renormalize=True):
    out = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        places = [j for j in range(indices.shape[1]) if indices[t, j] >= 0]
        if renormalize:
            over = [int(indices[t, j]) for j in places]
        else:
            over = [e for e in range(logits.shape[1]) if logits[t, e] != -math.inf]
        if not over:
            continue
        high = max(float(logits[t, e]) for e in over)
        total = sum(math.exp(float(logits[t, e]) - high) for e in over)
        g = {int(indices[t, j]): float(dweights[t, j]) for j in places}
        p = {e: math.exp(float(logits[t, e]) - high) / total for e in over}
        dot = sum(p[e] * v for e, v in g.items())
        for e in over:
            out[t, e] = p[e] * (g.get(e, 0.0) - dot)
    return out


def dispatch(x, indices, experts):
    """(xs, slot, offsets)"""
    tokens, top_k = indices.shape
    rows = [[] for _ in range(experts)]
    for t in range(tokens):
        for j in range(top_k):
            if 0 <= indices[t, j] < experts:
                rows[int(indices[t, j])].append((t, j))
    xs = np.zeros((tokens * top_k, x.shape[1]))
    slot = np.full((tokens, top_k), -1, dtype=np.int32)
    offsets = np.zeros(experts + 1, dtype=np.int32)
    at = 0
    for e in range(experts):
        for t, j in rows[e]:
            slot[t, j] = at
            xs[at] = x[t]
            at += 1
        offsets[e + 1] = at
    return xs, slot, offsets


def combine(ys, slot, weights=None, r=None):
    y = np.zeros((slot.shape[0], ys.shape[1])) if r is None else np.array(r, dtype=np.float64)
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            if slot[t, j] >= 0:
                y[t] += ys[slot[t, j]] * (1.0 if weights is None else float(weights[t, j]))
    return y


def combine_backward(dy, ys, slot, weights):
    """(dys, dweights)"""
    dys, dwts = np.zeros_like(ys), np.zeros(slot.shape)
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            if slot[t, j] >= 0:
                dys[slot[t, j]] = float(weights[t, j]) * dy[t]
                dwts[t, j] = ys[slot[t, j]] @ dy[t]
    return dys, dwts
