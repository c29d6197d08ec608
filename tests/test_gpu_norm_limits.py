"""Rows whose sums leave the range of fp32, as the header states it."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [100, 700, 1001, 4096, 9000, 40000, 40001])
def test_sums_beyond_the_largest_number(width, dtype):
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(3, width, generator=g, device="cuda")
    x[0] *= 1e25  # squares of 1e50
    x[1] = 3e38
    x = x.to(dtype)
    b = torch.randn(width, generator=g, device="cuda").to(dtype)
    y, mean, rstd = muon.layer_norm(x, bias=b, keep_stats=True)
    assert rstd[0] == 0 and torch.isfinite(mean[0]) and torch.equal(y[0], b)
    assert mean[1] == float("inf")
    assert torch.equal(y[2:], muon.layer_norm(x[2:].contiguous(), bias=b)) and torch.isfinite(y[2]).all()
    muon.check_ops_error()
