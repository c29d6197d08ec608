"""The layer operators' C ABI on the host: the library exports what the header
declares, and every argument error is a status before anything is launched."""
import ctypes as C
import os
import re

import pytest

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


def test_exports_every_declared_symbol(lib):
    hdr = open(os.path.join(ROOT, "include", "muon_ops.h"), encoding="utf-8").read()
    declared = set(re.findall(r"^MUON_API\s+muon_status_t\s+(muon_[a-z_0-9]+)\s*\(", hdr, re.M))
    assert declared == set(_capi.EXPORTED_OPS)
    for name in declared:
        assert hasattr(lib, name), name
    for name in ("MUON_MAX_EXPERTS", "MUON_MAX_TOP_K"):
        assert int(re.search(rf"#define {name} (\d+)", hdr).group(1)) == getattr(_capi, name)


def _args(**kw):
    a = _capi.muon_linear_args()
    base = {"dtype": 2, "rows": 8, "in": 16, "out": 24, "x_stride": 16, "w_stride": 24, "residual_stride": 24,
            "dy_stride": 24, "x": P, "w": P, "y": P, "dy": P, "dx": P, "dw": P}
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


BAD = [dict(dtype=3), dict(dtype=-1), dict(activation=5), dict(activation=-1), dict(w_layout=2), dict(experts=-1),
       dict(experts=1025, offsets=P), dict(rows=-1), dict(rows=(1 << 30) + 1), {"in": 0}, dict(out=0),
       dict(x_stride=15), dict(w_stride=23), dict(w_layout=1, w_stride=15), dict(x_stride=1 << 40),
       dict(experts=2), dict(experts=2, offsets=P, w_expert_stride=16 * 24 - 1)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: ",".join(f"{k}={v}" for k, v in b.items()))
def test_linear_refuses(lib, bad):
    n = C.c_size_t()
    a = _args(**bad)
    assert lib.muon_linear(C.byref(a), None) == INVALID
    assert lib.muon_linear_backward(C.byref(a), None) == INVALID
    assert lib.muon_linear_workspace(C.byref(a), 0, C.byref(n)) == INVALID
    assert lib.muon_last_error().decode().startswith("muon_linear")


def test_linear_refuses_null_pointers(lib):
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(residual=P, residual_stride=3)):
        assert lib.muon_linear(C.byref(_args(**kw)), None) == INVALID
    for kw in (dict(dy=None), dict(w=None), dict(x=None), dict(dx=None, dw=None), dict(activation=1),
               dict(dy_stride=23)):
        assert lib.muon_linear_backward(C.byref(_args(**kw)), None) == INVALID
    assert lib.muon_linear(None, None) == INVALID and lib.muon_linear_backward(None, None) == INVALID
    assert lib.muon_linear_workspace(C.byref(_args()), 0, None) == INVALID
    huge = {"rows": 1 << 30, "in": 1 << 20, "out": 1 << 20, "x_stride": 1 << 20, "w_stride": 1 << 20}
    assert lib.muon_linear(C.byref(_args(**huge)), None) == UNSUPPORTED


def test_linear_refuses_a_short_workspace(lib):
    a = _args(activation=2, preact=P, db=P)
    n = C.c_size_t()
    assert lib.muon_linear_workspace(C.byref(a), 1, C.byref(n)) == OK
    assert n.value > 0
    for ws, size in ((None, n.value), (P, n.value - 1), (P + 16, n.value)):
        a.workspace, a.workspace_bytes = ws, size
        assert lib.muon_linear_backward(C.byref(a), None) == INVALID
        assert "workspace" in lib.muon_last_error().decode()


def test_gate_refuses(lib):
    good = [0, 4, 16, 3, 1, P, 16, P, P, None]
    for i, v in ((0, 7), (1, -1), (2, 0), (2, 1025), (3, 0), (3, 17), (5, None), (6, 15), (7, None), (8, None)):
        bad = list(good)
        bad[i] = v
        assert lib.muon_gate(*bad) == INVALID, (i, v)
    good = [0, 4, 16, 3, 1, P, P, 16, P, P, None]
    for i, v in ((0, 7), (1, -1), (2, 0), (3, 17), (5, None), (6, None), (7, 15), (8, None), (9, None)):
        bad = list(good)
        bad[i] = v
        assert lib.muon_gate_backward(*bad) == INVALID, (i, v)
    assert lib.muon_gate(0, 0, 16, 3, 1, None, 16, None, None, None) == OK  # no tokens: nothing to do


def test_sort_refuses(lib):
    n = C.c_size_t()
    assert lib.muon_dispatch_workspace(4, 2, 8, C.byref(n)) == OK and n.value == 0  # few: one launch, no scratch
    assert lib.muon_dispatch_workspace(40000, 2, 8, C.byref(n)) == OK and n.value > 0
    for t, k, e in ((-1, 2, 8), (4, 0, 8), (4, 33, 8), (4, 2, 0), (4, 2, 1025), (1 << 30, 4, 8)):
        assert lib.muon_dispatch_workspace(t, k, e, C.byref(n)) == INVALID
    lib.muon_dispatch_workspace(40000, 2, 8, C.byref(n))
    good = [2, 40000, 16, 2, 8, P, 16, P, 32, P, P, P, P, n.value, None]
    for i, v in ((0, 9), (1, -1), (2, 0), (3, 0), (4, 0), (5, None), (6, 15), (7, None), (8, 16), (10, None),
                 (11, None), (12, None), (12, P + 8), (13, n.value - 1)):
        bad = list(good)
        bad[i] = v
        assert lib.muon_dispatch(*bad) == INVALID, (i, v)
    good = [2, 4, 16, 2, P, 16, P, P, None]
    for i, v in ((0, 9), (1, -1), (2, 0), (3, 33), (4, None), (5, 15), (6, None), (7, None)):
        bad = list(good)
        bad[i] = v
        assert lib.muon_dispatch_backward(*bad) == INVALID, (i, v)
    good = [2, 4, 16, 2, P, 16, P, P, P, 16, P, None]
    for i, v in ((0, 9), (3, 0), (4, None), (5, 15), (6, None), (7, None), (9, 15), (10, None)):
        bad = list(good)
        bad[i] = v
        assert lib.muon_combine(*bad) == INVALID, (i, v)
    good = [2, 4, 16, 2, 8, P, 16, P, 16, P, P, P, P, P, None]
    for i, v in ((0, 9), (4, 0), (5, None), (6, 15), (7, None), (8, 15), (9, None), (10, None), (11, None),
                 (12, None), (13, None)):
        bad = list(good)
        bad[i] = v
        assert lib.muon_combine_backward(*bad) == INVALID, (i, v)


def test_header_compiles_as_c(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    src = tmp_path / "ops.c"
    src.write_text('#include "muon_ops.h"\nint main(void) { muon_linear_args a = {0}; return (int)a.rows; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-Wno-missing-field-initializers",
                        "-I", os.path.join(ROOT, "include"), "-fsyntax-only", str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_argument_structure_matches_the_header():
    hdr = open(os.path.join(ROOT, "include", "muon_ops.h"), encoding="utf-8").read()
    body = re.search(r"typedef struct \{(.*?)\} muon_linear_args;", hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for decl in body.split(";") if decl.strip()
             for n in re.sub(r"^\s*(const\s+)?\w+", "", decl.strip()).split(",")]
    assert names == [f[0] for f in _capi.muon_linear_args._fields_]
