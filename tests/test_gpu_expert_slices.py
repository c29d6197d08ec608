"""Some of an expert tensor's experts: offsets that do not start at 0, as a slice
of all experts' offsets has them."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

from layers_tol import check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [[40, 75, 75, 139], [130, 200, 300, 420], [5, 5, 5, 5], [500, 500, 500, 500]],
                         ids=lambda o: "-".join(map(str, o)))
@pytest.mark.parametrize("rows", [150, 500])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_rows_before_the_first_range_belong_to_no_expert(dtype, rows, off):
    if off[-1] > rows:
        off = [min(o, rows) for o in off]
    g = torch.Generator(device="cuda").manual_seed(rows + off[0])
    x, dy, z = (torch.randn(rows, n, generator=g, device="cuda").to(dtype) for n in (72, 136, 136))
    w = (torch.randn(3, 72, 136, generator=g, device="cuda") / 8).to(dtype)
    b = torch.randn(3, 136, generator=g, device="cuda").to(dtype)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    held = [torch.full((rows, n), 7.0, dtype=dtype, device="cuda") for n in (136, 136, 72)]
    del held  # outputs are likely to be made from this memory: rows left out would show
    y, zz = muon.expert_linear(x, o, w, bias=b, activation="silu", keep_preact=True)
    dx, dw, db = muon.expert_linear_backward(dy, x, o, w, preact=z, activation="silu", bias=True)
    muon.check_ops_error()
    for t in (y, zz, dx):
        assert not t[:off[0]].any() and not t[off[-1]:].any()
    s = slice(off[0], rows)
    moved = [v - off[0] for v in off]
    if rows > off[0]:
        check_forward(y[s], zz[s], x[s], w, b, "silu", None, moved)
        check_backward((dx[s], dw, db), dy[s], x[s], w, z[s], "silu", moved)
    else:
        assert not dw.any() and not db.any()
