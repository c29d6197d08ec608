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


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd)"""
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_backward(dy, x, mean, rstd, w=None, r=None):
    """(dx, dw, db)"""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    return (dx if r is None else dx + r), (dy * xh).sum(axis=0), dy.sum(axis=0)


def balance_loss(logits, indices, coef=1.0):
    """(loss, counts, live)"""
    tokens, experts = logits.shape
    counts = np.zeros(experts, dtype=np.int32)
    for e in indices.reshape(-1):
        if 0 <= e < experts:
            counts[e] += 1
    live, mass = 0, np.zeros(experts)
    for t in range(tokens):
        open_ = logits[t] != -math.inf
        if open_.any():
            live += 1
            p = np.exp(logits[t][open_] - logits[t][open_].max())
            mass[open_] += p / p.sum()
    share = counts / max(int(counts.sum()), 1)
    return coef * experts * float((share * mass).sum()) / max(live, 1), counts, live


def balance_loss_backward(dloss, logits, counts, live, coef=1.0, r=None):
    out = np.zeros(logits.shape) if r is None else np.array(r, dtype=np.float64)
    share = counts / max(int(counts.sum()), 1)
    for t in range(logits.shape[0]):
        open_ = logits[t] != -math.inf
        if not open_.any():
            continue
        p = np.exp(logits[t][open_] - logits[t][open_].max())
        p /= p.sum()
        f = share[open_]
        out[t][open_] += dloss * coef * logits.shape[1] / max(live, 1) * p * (f - (p * f).sum())
    return out


MX_GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_round(x):
    """(values of x as microscaled 4-bit numbers, scale bytes): blocks of 32 along the
    last axis, each scaled by the power of two at or below its largest magnitude, over
    4, and rounded to the nearest of MX_GRID, ties to the even code."""
    *lead, n = x.shape
    blocks = -(-n // 32)
    rows = np.zeros((int(np.prod(lead, dtype=np.int64)), 32 * blocks))
    rows[:, :n] = np.asarray(x, dtype=np.float64).reshape(-1, n)
    rows = rows.reshape(-1, blocks, 32)
    scales = np.zeros(rows.shape[:2], dtype=np.uint8)
    out = np.zeros_like(rows)
    for i in range(rows.shape[0]):
        for b in range(blocks):
            block = rows[i, b]
            if not np.isfinite(block).all():
                scales[i, b], out[i, b] = 255, math.nan
                continue
            top = float(np.abs(block).max())
            e = -127 if top == 0.0 else min(max(math.frexp(top)[1] - 1 - 2, -127), 127)
            scales[i, b] = e + 127
            a = np.abs(block) / 2.0 ** e
            gap = np.abs(a[:, None] - MX_GRID)
            near = gap == gap.min(axis=1, keepdims=True)
            code = np.where(near.sum(axis=1) > 1, 2 * (near.argmax(axis=1) // 2 + near.argmax(axis=1) % 2), near.argmax(axis=1))
            out[i, b] = np.sign(block) * MX_GRID[code] * 2.0 ** e
    return out.reshape(-1, 32 * blocks)[:, :n].reshape(*lead, n), scales.reshape(*lead, blocks)


def mx_held(values, scales, n):
    """The numbers that packed bytes [.., 16 * blocks] and scale bytes [.., blocks] stand for."""
    v = np.stack((values & 15, values >> 4), axis=-1).reshape(*values.shape[:-1], -1)
    x = np.where(v & 8, -1.0, 1.0) * MX_GRID[v & 7]
    factor = np.where(scales == 255, math.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (x * np.repeat(factor, 32, axis=-1))[..., :n]
