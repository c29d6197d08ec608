"""Static checks of the layer operators' kernel sources."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_bucket_gb300", "csrc")


def _code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path, encoding="utf-8").read(), flags=re.S)


def test_programmatic_kernels_use_no_non_coherent_loads():
    """A kernel that may be resident while the launch before it writes its inputs
    reads them by ordinary loads only."""
    early = [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "grid_wait()" in _code(f)]
    assert len(early) >= 5
    for f in early:
        found = re.search(r"__ldg\b|ld\.global\.nc|__restrict__|\bld_hint\b", _code(f))
        assert not found, f"{os.path.basename(f)}: {found.group(0)}"


def test_programmatic_kernels_wait_for_the_launch_before():
    """Every kernel of a file that launches programmatically calls grid_wait."""
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        code = _code(f)
        if "grid_wait()" not in code:
            continue
        kernels = re.split(r"\b__global__\b", code)[1:]
        assert kernels and all("grid_wait()" in k for k in kernels), os.path.basename(f)


def test_stores_handed_to_the_other_cta_are_acquired_there():
    """The zeros behind a range's end are ordinary stores that the other CTA's MMAs
    read: released at cluster scope, and acquired at cluster scope before them."""
    code = _code(os.path.join(CSRC, "k_linear_tc.cu"))
    assert "mbar_arrive_release_cluster(map_to(full(st), 0))" in code
    issuer = code[code.index("umma_pair(d_tmem") - 1200:code.index("umma_pair(d_tmem")]
    assert "mbar_acquire_cluster(full(s), ph)" in issuer
    assert "acquire.cluster" in _code(os.path.join(CSRC, "mbarrier.cuh"))
