"""SiLU and the tanh form of GELU at every number of the 16-bit types, in each kernel
that applies them: weights of zero, so that a feature's pre-activation is its bias.

Both are z p with p = 1 / (1 + 2^t), t = -w log2(e), w = z or 2 sqrt(2/pi) (z + 0.044715
z^3).  w is off by at most 4.5 roundings of 2^-24 (none for z itself), t by one more
and the constant's, which 2^t turns into (1.2 + 4.5) |w| 2^-24 of itself; the hardware's
power of two is within 2^-22 and its reciprocal within 2^-23 of themselves, the sum
and the product are rounded once.  p below 2^-126 may come out as 0."""
import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

from layers_tol import U

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # of numbers below the smallest normal one


def _linear(z, rows):
    w = torch.zeros(64, z.numel(), dtype=z.dtype, device="cuda")
    return lambda kind: muon.linear(torch.zeros(rows, 64, dtype=z.dtype, device="cuda"), w, bias=z, activation=kind)


def _experts(z, rows):
    w = torch.zeros(1, 64, z.numel(), dtype=z.dtype, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    return lambda kind: muon.expert_linear(torch.zeros(rows, 64, dtype=z.dtype, device="cuda"), off, w, bias=z[None],
                                           activation=kind)


def _mx(z, rows):
    held = muon.mx_quantize(torch.zeros(64, z.numel(), dtype=z.dtype, device="cuda"))
    return lambda kind: muon.mx_linear(torch.zeros(rows, 64, dtype=z.dtype, device="cuda"), *held, bias=z, activation=kind)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("op,rows", [(_linear, 5), (_linear, 70), (_experts, 33), (_mx, 5), (_mx, 40), (_mx, 70)],
                         ids=["few", "tiles", "experts", "mx-few", "mx-narrow", "mx-tiles"])
def test_every_16_bit_value(op, rows, dtype):
    z = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(DT[dtype])
    run = op(z, rows)
    Z = z.double().cpu().numpy()
    for kind, steps in (("silu", 1.3), ("gelu_tanh", 6.0)):
        y = run(kind)
        assert torch.equal(y.view(torch.int16), y[:1].view(torch.int16).expand_as(y))  # every token's
        got = y[0].double().cpu().numpy()
        with np.errstate(all="ignore"):
            w = Z if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (Z + 0.044715 * Z ** 3)
            want = Z / (1 + np.exp(-w))
            want[np.isneginf(Z)] = np.nan  # -infinity times 0
            assert np.array_equal(np.isnan(got), np.isnan(want))
            live = np.isfinite(want)
            assert np.array_equal(got[~live & ~np.isnan(want)], want[~live & ~np.isnan(want)])
            tol = (steps * np.minimum(np.abs(w), 100) + 12) * 2.0 ** -24 * np.abs(want) + 1.01 * 2.0 ** -126 * np.abs(Z)
            tol = tol + 1.01 * U[DT[dtype]] * (np.abs(want) + tol) + HALF_STEP[dtype]
            bad = live & ~(np.abs(got - want) <= tol)
        assert not bad.any(), (kind, Z[bad][:3], got[bad][:3], want[bad][:3])
    muon.check_ops_error()
