"""Tensors of more than 2^31 elements through the layer norm, the balance loss and the
4-bit operators: element offsets do not fit in 32 bits.  Rows at the start, the
middle and the end are checked."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon

from layers_tol import U, acc

pytestmark = pytest.mark.gpu


def _need(gib):
    if torch.cuda.mem_get_info()[0] < gib * (1 << 30):
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("rows,width", [(530000, 4104), (2200000, 1001)])
def test_layer_norm_past_32_bits(rows, width):
    _need(32)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, width, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(width, generator=g, device="cuda")
    y, mean, rstd = muon.layer_norm(x, w, keep_stats=True)
    pick = torch.tensor([0, 1, rows // 2, (1 << 31) // width, (1 << 31) // width + 1, rows - 1], device="cuda")
    d = x[pick].double()
    want = torch.nn.functional.layer_norm(d, (width,), w.double())
    assert ((y[pick].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-4).all()
    del y
    dy = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    dy[pick] = 0.5
    dx, dw, db = muon.layer_norm_backward(dy, x, mean, rstd, w, bias=True)
    assert torch.equal(db, torch.full_like(db, 0.5 * len(pick)))
    xh = (d - d.mean(1, keepdim=True)) * (d.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    assert ((dw.double() - 0.5 * xh.sum(0)).abs() <= 1e-4).all()
    gw = 0.5 * w.double()
    want = (d.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * (gw - gw.mean() - xh * (gw * xh).mean(1, keepdim=True))
    assert ((dx[pick].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 1e-4).all()
    dx[pick] = 0
    assert not dx.any()


def test_balance_loss_past_32_bits():
    _need(24)
    tokens, experts = 2200000, 1000
    logits = torch.zeros(tokens, experts, dtype=torch.bfloat16, device="cuda")
    idx = (torch.arange(tokens, device="cuda", dtype=torch.int32) % experts)[:, None].contiguous()
    loss, counts, live = muon.balance_loss(logits, idx)
    assert int(live) == tokens and torch.equal(counts, torch.full_like(counts, tokens // experts))
    assert abs(float(loss) - 1) <= acc(1000) + acc(400)
    logits[-1, 0] = 3.0  # the last token alone has a gradient: its expert is as busy as the others, so that it is 0 too
    counts[0] += 1000
    d = muon.balance_loss_backward(torch.full((), 1e6, device="cuda"), logits, counts, live)
    last = logits[-1:].double().requires_grad_()
    share = counts.double() / counts.sum()
    (1e6 * experts / tokens * (torch.softmax(last, 1) * share).sum()).backward()
    assert ((d[-1:].double() - last.grad).abs() <= 2.0 ** -8 * 1.01 * last.grad.abs() + 1e-9).all()
    assert torch.equal(d[0], d[tokens // 2])


def test_mx_products_past_32_bits():
    _need(24)
    rows, n_in, n_out = 70001, 72, 40008
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, n_in, generator=g, device="cuda").bfloat16()
    values, scales = muon.mx_quantize(torch.randn(n_in, n_out, generator=g, device="cuda"))
    w = muon.mx_dequantize(values, scales, n_in, dtype=torch.float32).double()
    y = muon.mx_linear(x, values, scales, activation="relu")
    muon.check_ops_error()
    pick = torch.tensor([0, 1, 26843, 53687, 53688, rows - 2, rows - 1], device="cuda")
    xq = muon.mx_dequantize(*muon.mx_quantize(x[pick].t()), n_in, dtype=torch.float32).t().double()
    want = (xq @ w).clamp(min=0)
    tol = acc(n_in) * (xq.abs() @ w.abs()) + U[torch.bfloat16] * 1.01 * want + 1e-37
    assert ((y[pick].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("out_in", [False, True])
def test_mx_weights_past_32_bits(out_in):
    _need(32)
    experts, n_in, n_out = 5, 33000, 13120
    g = torch.Generator(device="cuda").manual_seed(3)
    shape = (experts, n_out, n_in) if out_in else (experts, n_in, n_out)
    w = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)
    w = w.transpose(-1, -2) if out_in else w
    values, scales = muon.mx_quantize(w)
    back = muon.mx_dequantize(values, scales, n_in)
    for e, cols in ((0, slice(0, 40)), (2, slice(6000, 6050)), (experts - 1, slice(n_out - 40, n_out))):
        v, s = muon.mx_quantize(w[e][:, cols].contiguous())
        assert torch.equal(values[e, cols], v) and torch.equal(scales[e, cols], s)
        assert torch.equal(back[e][:, cols], muon.mx_dequantize(v, s, n_in))
