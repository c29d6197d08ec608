"""Products of 4-bit operands whose sums are longer than a kernel's ring of stages, so
that every stage, and every set of scale columns, is used again: within a tile, and
from one tile to the next.  Which form a product takes follows from its sizes:
  one matrix, up to 16 rows    clusters that share the sum and round the rows themselves
  17 .. 64 rows, out <= 9728   the same behind the rounding launch (4 or 5 stages)
  17 .. 64 rows, wider         tiles of 64 rows (9 stages, as many sets of scales)
  experts                      tiles of 64, 128 or 192 rows for up to 32, 64 or more an expert"""
import numpy as np
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from oracle import layers_ref as ref

from layers_tol import check_forward, to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _randn(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _weights(shape, seed):
    """Packed weights, and the numbers that they stand for as [.., in, out] in 64 bits."""
    values, scales = muon.mx_quantize(_randn(shape, torch.bfloat16, seed, shape[-2] ** -0.5))
    held = ref.mx_held(values.cpu().numpy(), scales.cpu().numpy(), shape[-2])
    return values, scales, torch.from_numpy(held).transpose(-1, -2)


def _rounded(x):
    return torch.from_numpy(ref.mx_round(to64(x))[0])


# (rows, in, out): shares of the sum of 8 stages and more, an odd rest of the last one; then tiles of 64 rows
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", [(16, 16384, 130), (3, 20000, 257), (17, 16384, 129), (33, 16384, 300), (48, 11000, 128),
                                  (64, 16420, 200), (64, 8192, 1300), (40, 2600, 9800), (64, 5003, 9729)],
                         ids=lambda c: "x".join(map(str, c)))
def test_few_rows_of_a_long_sum(case, dtype):
    rows, n_in, n_out = case
    x = _randn((rows, n_in), DT[dtype], 1)
    values, scales, W = _weights((n_in, n_out), 2)
    b, r = _randn((n_out,), DT[dtype], 3), _randn((rows, n_out), DT[dtype], 4)
    y = muon.mx_linear(x, values, scales, bias=b, activation="silu", residual=r)
    muon.check_ops_error()
    check_forward(y, None, _rounded(x), W, b, "silu", r)
    assert all(torch.equal(muon.mx_linear(x, values, scales, bias=b, activation="silu", residual=r), y) for _ in range(3))


def test_few_rows_share_a_sum_four_ways():
    """64 rows that fill the GPU with clusters of four, eight stages each."""
    x = _randn((64, 8192), torch.bfloat16, 1)
    values, scales, W = _weights((8192, 8192), 2)
    y = muon.mx_linear(x, values, scales)
    muon.check_ops_error()
    check_forward(y, None, _rounded(x), W, None, "none", None)


# rows of each range; the average decides on the tiles' rows
EXPERTS = {
    64: [63, 64, 65, 129, *(n for n in (1, 0, 31, 32, 33, 7, 18, 20, 2, 16, 24, 9) for _ in range(2))],
    128: [127, 128, 129, 193, 1, 0, 64, 65, 33, 2, 31, 40, 63, 50, 5, 20],
    192: [191, 192, 193, 385, 1, 0, 100, 64, 65, 70, 129, 300],
}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tile", list(EXPERTS))
def test_experts_of_a_long_sum(tile, dtype):
    """20 stages a tile and more tiles than pairs of SMs, for each number of rows a tile."""
    sizes = EXPERTS[tile]
    experts, rows = len(sizes), sum(sizes)
    each = -(-rows // min(rows, experts))
    assert (64 if each <= 32 else 128 if each <= 64 else 192) == tile
    n_in, n_out = 5024, {64: 776, 128: 1100, 192: 1400}[tile]
    assert sum(-(-n // tile) for n in sizes) * -(-n_out // 256) > 76
    x = _randn((rows + 5, n_in), DT[dtype], 1)
    values, scales, W = _weights((experts, n_in, n_out), 2)
    ends = [0, *np.cumsum(sizes).tolist()]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    b = _randn((experts, n_out), DT[dtype], 3)
    y = muon.mx_expert_linear(x, off, values, scales, bias=b, activation="relu")
    muon.check_ops_error()
    assert not y[rows:].any()
    check_forward(y[:rows], None, _rounded(x[:rows]), W, b, "relu", None, ends)
    assert all(torch.equal(muon.mx_expert_linear(x, off, values, scales, bias=b, activation="relu"), y) for _ in range(3))
