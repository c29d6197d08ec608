"""A norm's block whose wait for a row runs out ends: it stores nothing from that row
on, the other blocks finish, the error word tells, and the context stays usable.
Nothing here faults or hangs: the barrier of one slot of one block's ring expects one
arrival more than it gets, and the wait for it gives up after half a millisecond."""
import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from newton_schulz_bucket_gb300 import _capi

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, _capi.MUON_DTYPE_BF16), "fp16": (torch.float16, _capi.MUON_DTYPE_F16),
      "fp32": (torch.float32, _capi.MUON_DTYPE_F32)}
LIMIT = 1 << 20
MARK = 77.0


def _lost(dtype, x, block, slot, dy=None, mean=None, rstd=None, out=None, dw=None):
    p = [None if t is None else t.data_ptr() for t in (x, dy, mean, rstd, out, dw)]
    torch.cuda.synchronize()
    return _capi.load().muon_testing_norm_lost_row(DT[dtype][1], *x.shape, block, slot, LIMIT, *p, None)


def _inputs(rows, width, dtype):
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randn(rows, width, generator=g, device="cuda").to(DT[dtype][0])
    return x, torch.randn(rows, width, generator=g, device="cuda").to(DT[dtype][0])


def _gone(stored):
    gone = (~stored).nonzero()[:, 0].tolist()
    return gone, {b - a for a, b in zip(gone, gone[1:])}


# blocks with 16 and 32 elements a thread, one to many an SM, whole pieces and single elements: in each, three
# rows to a block at least but for the last
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,width", [(6000, 520), (4000, 4096), (6000, 1001), (2000, 8192), (700, 12001), (1000, 16384), (3, 4096)])
def test_forward(rows, width, dtype):
    x, _ = _inputs(rows, width, dtype)
    want = muon.layer_norm(x, keep_stats=True)
    muon.check_ops_error()
    for block, slot in ((0, 0), (2, 0), (100, 1), (151, 2)) if rows > 3 else ((0, 0), (2, 0)):
        y = torch.full_like(x, MARK)
        mean, rstd = (torch.full((rows,), MARK, device="cuda") for _ in range(2))
        assert _lost(dtype, x, block, slot, mean=mean, rstd=rstd, out=y) == _capi.MUON_ERR_TIMEOUT
        stored = mean != MARK
        gone, apart = _gone(stored)  # each grid's size of rows one
        assert len(apart) <= 1 and 0 < len(gone) < rows
        d = min(apart, default=rows)
        assert gone[0] == block + (slot * d if rows > 3 else 0) and gone[-1] + d >= rows
        assert torch.equal(stored, rstd != MARK) and (y[~stored] == MARK).all()
        assert all(torch.equal(got[stored], w[stored]) for got, w in zip((y, mean, rstd), want))
    y = torch.full_like(x, MARK)
    assert _lost(dtype, x, rows + 1, 0, out=y) == _capi.MUON_OK and torch.equal(y, want[0])  # no such block
    again = muon.layer_norm(x, keep_stats=True)
    assert all(torch.equal(p, q) for p, q in zip(again, want))
    muon.check_ops_error()


# rows in registers, and held in the ring
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,width", [(6000, 520), (4000, 4096), (3000, 1001), (2000, 8192), (900, 12001), (1000, 16384), (3, 9000)])
def test_backward(rows, width, dtype):
    x, dy = _inputs(rows, width, dtype)
    _, mean, rstd = muon.layer_norm(x, keep_stats=True)
    want = muon.layer_norm_backward(dy, x, mean, rstd)
    for block, slot in ((0, 0), (2, 0), (100, 0), (57, 1)) if rows > 3 else ((0, 0), (2, 0)):
        if slot and 3 * x[0].nbytes + 48 > 104 * 1024:
            continue  # (a ring of one slot)
        dx, dw = torch.full_like(x, MARK), torch.empty(width, dtype=x.dtype, device="cuda")
        assert _lost(dtype, x, block, slot, dy, mean, rstd, dx, dw) == _capi.MUON_ERR_TIMEOUT
        stored = (dx != MARK).any(dim=1)
        gone, apart = _gone(stored)  # the rest of the block's part of rows
        assert apart <= {1} and 0 < len(gone) < rows
        assert (dx[~stored] == MARK).all() and torch.equal(dx[stored], want[0][stored])
        part = len(gone) + slot
        assert gone[0] == block * part + slot or gone[-1] == rows - 1
        assert _lost(dtype, x, block, slot, dy, mean, rstd, None, dw) == _capi.MUON_ERR_TIMEOUT  # dw alone
    again = muon.layer_norm_backward(dy, x, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(again[:2], want[:2]))
    muon.check_ops_error()


def test_the_next_kernels_are_whole():
    """Norms that follow at once on the same SMs."""
    x, _ = _inputs(2000, 4096, "bf16")
    want = muon.layer_norm(x)
    y = torch.empty_like(x)
    for i in range(3):
        assert _lost("bf16", x, i, 1, out=y) == _capi.MUON_ERR_TIMEOUT
        got = [muon.layer_norm(x) for _ in range(4)]
        assert all(torch.equal(t, want) for t in got)
    muon.check_ops_error()


def test_refusals():
    x, dy = _inputs(4, 1024, "bf16")
    y = torch.empty_like(x)
    one = torch.zeros(4, device="cuda")
    L = _capi.load()
    p = lambda t: t.data_ptr()  # noqa: E731
    for args in ((2, 4, 512, 0, 0, LIMIT, p(x), None, None, None, p(y), None, None),
                 (2, 4, 16385, 0, 0, LIMIT, p(x), None, None, None, p(y), None, None),
                 (2, 4, 1024, -1, 0, LIMIT, p(x), None, None, None, p(y), None, None),
                 (2, 4, 1024, 0, 8, LIMIT, p(x), None, None, None, p(y), None, None),
                 (2, 4, 1024, 0, -1, LIMIT, p(x), None, None, None, p(y), None, None),
                 (2, 4, 1024, 0, 0, 1023, p(x), None, None, None, p(y), None, None),
                 (7, 4, 1024, 0, 0, LIMIT, p(x), None, None, None, p(y), None, None),
                 (2, 4, 1024, 0, 0, LIMIT, None, None, None, None, p(y), None, None),
                 (2, 4, 1024, 0, 0, LIMIT, p(x), None, None, None, None, None, None),
                 (2, 4, 1024, 0, 0, LIMIT, p(x), p(dy), None, p(one), p(y), None, None),
                 (2, 4, 1024, 0, 0, LIMIT, p(x), p(dy), p(one), p(one), None, None, None)):
        assert L.muon_testing_norm_lost_row(*args) == _capi.MUON_ERR_INVALID_ARG
