"""Element-wise error bounds of the layer operators, from their arithmetic.

u: unit roundoff of the store.  A sum of n fp32 terms, in any order and with
adds that truncate, is within (n + 16) 2^-23 of the sum of magnitudes.  The
activations' slopes stay below 1.2 and their fp32 evaluations (hardware
exponential and division included) within 2^-19 (1 + |z|).  dz is rounded to
the operand type before its two products.
"""
import numpy as np
import torch

from oracle import layers_ref as ref

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}


def to64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def acc(n):
    return (n + 16) * 2.0 ** -23


def close(got, want, tol, what):
    got = to64(got)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(int(np.argmax(bad)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {tuple(map(int, i))}: "
                             f"{got[i]!r} vs {want[i]!r}, tolerance {np.broadcast_to(tol, want.shape)[i]!r}")


def check_forward(y, z, x, w, b, kind, r, offsets=None):
    """y (and z) of linear or, with offsets, of expert_linear."""
    dt = y.dtype
    X, W = to64(x), to64(w)
    B = None if b is None else to64(b)
    R = None if r is None else to64(r)
    aB = None if b is None else np.abs(B)
    if offsets is None:
        Y, Z = ref.linear(X, W, B, kind, R)
        size = ref.linear(np.abs(X), np.abs(W), aB)[1]
    else:
        off = [int(v) for v in offsets]
        live = np.arange(X.shape[0]) < off[-1]
        X = np.where(live[:, None], X, 0)
        Y, Z = ref.expert_linear(X, off, W, B, kind, R)
        size = ref.expert_linear(np.abs(X), off, np.abs(W), aB)[1]
    dz = acc(X.shape[1]) * size
    tol = 1.2 * dz + 2.0 ** -19 * (1 + np.abs(Z)) * (kind != "none") + (0 if r is None else 2.0 ** -23 * np.abs(R))
    close(y, Y, tol + U[dt] * (np.abs(Y) + tol) * 1.01 + TINY[dt], "y")
    if z is not None:
        close(z, Z, dz + U[dt] * (np.abs(Z) + dz) * 1.01 + TINY[dt], "z")


def check_backward(got, dy, x, w, z, kind, offsets=None):
    dx, dw, db = got
    dt = x.dtype
    DY, X, W = to64(dy), to64(x), to64(w)
    Z = None if z is None else to64(z)
    off = None if offsets is None else [int(v) for v in offsets]
    if off is not None:
        live = (np.arange(X.shape[0]) < off[-1])[:, None]
        DY, X, Z = np.where(live, DY, 0), np.where(live, X, 0), None if Z is None else np.where(live, Z, 0)
        DX, DW, DB, DZ = ref.expert_linear_backward(DY, X, off, W, Z, kind)
        longest = max([b - a for a, b in zip(off, off[1:])] + [1])
    else:
        DX, DW, DB, DZ = ref.linear_backward(DY, X, W, Z, kind)
        longest = X.shape[0]
    e = np.zeros_like(DZ)  # error of dz: slope, and its rounding as an operand
    if kind != "none":
        e = 2.0 ** -18 * (1 + Z * Z) * np.abs(DY)
    op = e + (U[dt] * (np.abs(DZ) + e) + TINY[dt] if kind != "none" and dt != torch.float32 else 0)
    aDZ = np.abs(DZ) + op

    def back(d, xx, ww):
        if off is None:
            return ref.linear_backward(d, xx, ww)
        return ref.expert_linear_backward(d, xx, off, ww)

    eX, eW, _, _ = back(op, np.abs(X), np.abs(W))
    sX, sW, sB, _ = back(aDZ, np.abs(X), np.abs(W))
    eB = back(e, X, W)[2]
    if dx is not None:
        t = eX + acc(W.shape[-1]) * sX
        close(dx, DX, t + U[dt] * (np.abs(DX) + t) * 1.01 + TINY[dt], "dx")
    if dw is not None:
        t = eW + acc(longest) * sW
        close(dw, DW, t + U[dt] * (np.abs(DW) + t) * 1.01 + TINY[dt], "dw")
    if db is not None:
        t = eB + acc(longest) * sB
        close(db, DB, t + U[dt] * (np.abs(DB) + t) * 1.01 + TINY[dt], "db")
