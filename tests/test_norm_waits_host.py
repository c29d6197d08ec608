"""The refusals of the hook that makes a norm's wait run out: statuses before anything is
launched, so that no GPU is needed."""
import os

import pytest

from newton_schulz_bucket_gb300 import _capi

P = 4096  # a non-NULL pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.lib_path()):
        from newton_schulz_bucket_gb300 import build
        build.build()
    return _capi.load()


def test_norm_lost_row_refuses(lib):
    forward = [2, 4, 1024, 0, 0, 1 << 20, P, None, None, None, P, None, None]
    backward = [2, 4, 1024, 0, 0, 1 << 20, P, P, P, P, P, P, None]
    for good, more in ((forward, [(10, None), (11, P)]), (backward, [(8, None), (9, None)])):
        for i, v in [(0, 7), (1, 0), (1, (1 << 20) + 1), (2, 512), (2, 16385), (3, -1), (4, -1), (4, 8), (5, 1023),
                     (5, (1 << 33) + 1), (6, None), *more]:
            args = list(good)
            args[i] = v
            assert lib.muon_testing_norm_lost_row(*args) == _capi.MUON_ERR_INVALID_ARG, (i, v)
    backward[10] = backward[11] = None
    assert lib.muon_testing_norm_lost_row(*backward) == _capi.MUON_ERR_INVALID_ARG
