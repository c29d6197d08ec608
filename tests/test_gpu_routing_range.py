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


@pytest.mark.parametrize("n", [-1, -(1 << 32), (1 << 32) + 2, 1 << 31, 1 << 40])
def test_counts_that_no_32_bits_hold_are_refused(n):
    """Not taken for what their low 32 bits say, and before anything is allocated."""
    x = torch.zeros(4, 16, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(muon.MuonError, match="top_k"):
        muon.gate(x, n)
    with pytest.raises(muon.MuonError, match="experts"):
        muon.dispatch(x, idx, n)
    assert torch.cuda.max_memory_allocated() <= held + 4096
