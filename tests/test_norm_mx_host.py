"""The C ABI of the layer norm, the balance loss and microscaled weights on the host:
every argument error is a status before anything is launched; and the binding's
refusals, which need no GPU."""
import ctypes as C
import os
import re

import pytest
import torch

import newton_schulz_bucket_gb300 as muon
from newton_schulz_bucket_gb300 import _capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = _capi.MUON_OK, _capi.MUON_ERR_INVALID_ARG, _capi.MUON_ERR_UNSUPPORTED
P = 4096  # a non-NULL pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.lib_path()):
        from newton_schulz_bucket_gb300 import build
        build.build()
    return _capi.load()


def _refuses(call, good, bad, status=INVALID):
    for i, v in bad:
        args = list(good)
        args[i] = v
        assert call(*args) == status, (i, v)


def test_layer_norm_refuses(lib):
    good = [2, 0, 4, 16, 1e-5, P, 16, P, P, P, P, P, None]
    _refuses(lib.muon_layer_norm, good, [(0, 7), (1, 1), (2, -1), (2, (1 << 30) + 1), (3, 0), (3, (1 << 30) + 1),
                                         (4, -1e-5), (4, float("inf")), (4, float("nan")), (5, None), (6, 15),
                                         (6, 1 << 40), (9, None)])
    assert lib.muon_layer_norm(2, 0, 0, 16, 1e-5, None, 16, None, None, None, None, None, None) == OK
    n = C.c_size_t()
    assert lib.muon_layer_norm_workspace(4, 16, C.byref(n)) == OK and n.value > 0
    assert lib.muon_layer_norm_workspace(0, 16, C.byref(n)) == OK and n.value == 0
    assert lib.muon_layer_norm_workspace(4, 16, None) == INVALID
    assert lib.muon_layer_norm_workspace(4, 0, C.byref(n)) == INVALID
    lib.muon_layer_norm_workspace(4, 16, C.byref(n))
    good = [2, 2, 4, 16, P, 16, P, 16, P, P, P, P, 16, P, P, P, P, n.value, None]
    _refuses(lib.muon_layer_norm_backward, good,
             [(0, -1), (1, 1), (2, -1), (3, 0), (4, None), (5, 15), (6, None), (7, 15), (8, None), (9, None), (12, 15),
              (16, None), (16, P + 16), (17, n.value - 1)])
    good[13] = good[14] = good[15] = None
    assert lib.muon_layer_norm_backward(*good) == INVALID
    assert "all NULL" in lib.muon_last_error().decode()


def test_balance_loss_refuses(lib):
    n = C.c_size_t()
    assert lib.muon_balance_loss_workspace(100, 64, C.byref(n)) == OK and n.value == 0  # few: one launch, no scratch
    assert lib.muon_balance_loss_workspace(100000, 64, C.byref(n)) == OK and n.value > 0
    for t, e in ((-1, 64), (4, 0), (4, 1025)):
        assert lib.muon_balance_loss_workspace(t, e, C.byref(n)) == INVALID
    assert lib.muon_balance_loss_workspace(4, 16, None) == INVALID
    lib.muon_balance_loss_workspace(100000, 16, C.byref(n))
    good = [0, 100000, 16, 3, 1.0, P, 16, P, P, P, P, P, n.value, None]
    _refuses(lib.muon_balance_loss, good,
             [(0, 5), (1, -1), (2, 0), (3, 0), (3, 17), (4, float("nan")), (5, None), (6, 15), (7, None), (8, None),
              (9, None), (10, None), (11, None), (11, P + 8), (12, n.value - 1)])
    assert lib.muon_balance_loss(0, 1 << 30, 64, 3, 1.0, P, 64, P, P, P, P, P, 1 << 40, None) == INVALID
    good = [0, 4, 16, 1.0, P, P, 16, P, P, P, 16, P, None]
    _refuses(lib.muon_balance_loss_backward, good,
             [(0, 5), (1, -1), (2, 1025), (3, float("inf")), (4, None), (5, None), (6, 15), (7, None), (8, None), (10, 15),
              (11, None)])


def test_mx_quantize_refuses(lib):
    good = [2, 0, 2, 64, 24, P, 24, 64 * 24, P, P, None]
    _refuses(lib.muon_mx_quantize, good,
             [(0, 3), (1, 2), (2, -1), (2, 1025), (3, 0), (4, 0), (3, (1 << 30) + 1), (5, None), (6, 23), (6, 1 << 40),
              (7, 64 * 24 - 1), (7, 1 << 40), (8, None), (8, P + 8), (9, None)])
    assert lib.muon_mx_quantize(2, 1, 0, 64, 24, P, 63, 0, P, P, None) == INVALID  # rows of [out, in]
    assert lib.muon_mx_quantize(2, 0, 0, 1 << 30, 1 << 30, P, 1 << 30, 0, P, P, None) == UNSUPPORTED
    good = [2, 2, 64, 24, P, P, P, None]
    _refuses(lib.muon_mx_dequantize, good, [(0, 3), (1, -1), (2, 0), (3, 0), (4, None), (4, P + 4), (5, None), (6, None)])


def _args(**kw):
    a = _capi.muon_mx_linear_args()
    base = {"dtype": 2, "rows": 80, "in": 64, "out": 24, "x_stride": 64, "residual_stride": 24, "x": P, "w_values": P,
            "w_scales": P, "y": P, "workspace": P, "workspace_bytes": 1 << 30}
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


BAD = [dict(dtype=3), dict(activation=5), dict(activation=-1), dict(experts=-1), dict(experts=1025, offsets=P),
       dict(rows=-1), dict(rows=(1 << 30) + 1), {"in": 0}, dict(out=0), dict(x_stride=63), dict(x_stride=1 << 40),
       dict(residual=P, residual_stride=23)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_mx_linear_refuses(lib, bad):
    n = C.c_size_t()
    assert lib.muon_mx_linear(C.byref(_args(**bad)), None) == INVALID
    assert lib.muon_mx_linear_workspace(C.byref(_args(**bad)), C.byref(n)) == INVALID


def test_mx_linear_refuses_pointers_and_sizes(lib):
    for kw in (dict(x=None), dict(w_values=None), dict(w_scales=None), dict(y=None), dict(w_values=P + 8),
               dict(experts=2), dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=64)):
        assert lib.muon_mx_linear(C.byref(_args(**kw)), None) == INVALID, kw
    assert lib.muon_mx_linear(None, None) == INVALID
    n = C.c_size_t()
    assert lib.muon_mx_linear_workspace(C.byref(_args()), None) == INVALID
    assert lib.muon_mx_linear_workspace(C.byref(_args(rows=0)), C.byref(n)) == OK and n.value == 0
    huge = {"rows": 1 << 30, "in": 1 << 20, "out": 1 << 20, "x_stride": 1 << 20}
    assert lib.muon_mx_linear(C.byref(_args(**huge)), None) == UNSUPPORTED


@pytest.mark.parametrize("rows", [1, 64, 65, 1000, 100000])
@pytest.mark.parametrize("experts", [0, 1, 64])
def test_mx_workspace_holds_the_rounded_rows(lib, rows, experts):
    n = C.c_size_t()
    a = _args(rows=rows, experts=experts, **{"in": 1000, "x_stride": 1000})
    assert lib.muon_mx_linear_workspace(C.byref(a), C.byref(n)) == OK
    parts, mats = 8, max(experts, 1)
    if rows == 1 and not experts:  # few rows: one launch, no scratch
        assert n.value == 0
        return
    assert n.value >= rows * 32 * 17 + mats * 512 * parts
    assert n.value <= 3 * rows * 32 * 17 + mats * (512 * parts * 2 + 1024 * parts) + 2048


def test_argument_structure_matches_the_header():
    hdr = open(os.path.join(ROOT, "include", "muon_ops.h"), encoding="utf-8").read()
    body = re.search(r"typedef struct \{([^}]*)\} muon_mx_linear_args;", hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for decl in body.split(";") if decl.strip()
             for n in re.sub(r"^\s*(const\s+)?\w+", "", decl.strip()).split(",")]
    assert names == [f[0] for f in _capi.muon_mx_linear_args._fields_]


def test_the_binding_refuses_tensors_that_are_not_on_a_gpu_or_require_grad():
    x = torch.zeros(4, 64)
    f, i, u = torch.zeros(4), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, 32, dtype=torch.uint8)
    s, off = torch.zeros(8, 2, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    calls = [lambda x: muon.layer_norm(x), lambda x: muon.layer_norm_backward(x, x, f, f), lambda x: muon.balance_loss(x, i),
             lambda x: muon.balance_loss_backward(f[0], x, i[0], i[0, 0]), lambda x: muon.mx_quantize(x),
             lambda x: muon.mx_linear(x, u, s), lambda x: muon.mx_expert_linear(x, off, u[None], s[None])]
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call(x.clone().requires_grad_())
        with pytest.raises(ValueError, match="CUDA"):
            call(x)
    with pytest.raises(ValueError, match="CUDA"):
        muon.mx_dequantize(u, s, 64)
    with pytest.raises(ValueError, match="n_in"):
        muon.mx_dequantize(u, s, 0)
