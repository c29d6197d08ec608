"""Routing calls at the ends of their range."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden", [16, (1 << 22) + 3, (1 << 25) + 8])
def test_no_tokens_of_any_width(hidden):
    x = torch.empty(0, hidden, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    xs, slot, offsets = muon.dispatch(x, idx, 5)
    assert xs.shape == (0, hidden) and slot.shape == (0, 2) and offsets.tolist() == [0] * 6
