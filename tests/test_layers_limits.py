"""Which sizes the layer operators accept: whatever their launches can count."""
import ctypes as C
import os

import pytest

from newton_schulz_bucket_gb300 import _capi

P = 4096  # a non-NULL pointer that is not followed


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.lib_path()):
        from newton_schulz_bucket_gb300 import build
        build.build()
    return _capi.load()


def _size(lib, backward, rows, n_in, n_out, experts=0, dtype=2, **kw):
    a = _capi.muon_linear_args()
    a.dtype, a.rows, a.out, a.experts = dtype, rows, n_out, experts
    setattr(a, "in", n_in)
    a.x_stride, a.w_stride, a.residual_stride, a.dy_stride = n_in, n_out, n_out, n_out
    a.w_expert_stride = min(n_in * n_out, 1 << 36)
    for k in ("x", "w", "y", "dy", "dx", "dw", "db", "offsets"):
        setattr(a, k, P)
    for k, v in kw.items():
        setattr(a, k, v)
    n = C.c_size_t()
    return lib.muon_linear_workspace(C.byref(a), backward, C.byref(n)), n.value


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("size", [(3, (1 << 22) + 8, 16), (3, 16, (1 << 22) + 8), (1, 1 << 30, 1), (1, 1, 1 << 30),
                                  (1 << 30, 8, 8), (70, (1 << 24) + 8, 64), (1 << 20, 1 << 16, 8)])
@pytest.mark.parametrize("dtype", [0, 2])
def test_linear_accepts_what_memory_holds(lib, size, backward, dtype):
    assert _size(lib, backward, *size, dtype=dtype)[0] == _capi.MUON_OK
    if size[0] > 1:
        assert _size(lib, backward, *size, experts=2, dtype=dtype)[0] == _capi.MUON_OK


@pytest.mark.parametrize("size", [(1 << 30, 1 << 30, 1 << 30), (1, 1 << 30, 1 << 30), (1 << 30, 1 << 20, 1)])
def test_linear_refuses_what_no_launch_counts(lib, size):
    assert _size(lib, 0, *size)[0] == _capi.MUON_ERR_UNSUPPORTED
    assert _size(lib, 1, *size, experts=1024)[0] in (_capi.MUON_ERR_UNSUPPORTED, _capi.MUON_ERR_INVALID_ARG)


def test_expert_stride_of_huge_rows(lib):
    """(in - 1) * w_stride does not fit in 64 bits."""
    kw = dict(w_stride=1 << 36, w_expert_stride=1 << 20)
    assert _size(lib, 0, 4, 1 << 30, 8, experts=2, **kw)[0] == _capi.MUON_ERR_INVALID_ARG
