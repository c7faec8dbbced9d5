"""Kernels that are launched before their predecessor in the stream has ended read what it writes only after
pdl_wait(). A load through the non-coherent path (ld.global.nc) is taken to be of memory that nothing writes while the
kernel runs: the compiler may move it above the wait, and the cache may answer it with a line from before. So
nothing in the sources asks for one: no __ldg, no ld.global.nc, and no __restrict__ pointer, from which the
compiler may make one by itself. (No GPU.)"""
import glob
import os
import re

import matrix_dense_linear_spd_gb300 as bl

CSRC = os.path.join(os.path.dirname(bl.__file__), "csrc")


def code(path):
    """Without comments."""
    with open(path) as fh:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", fh.read(), flags=re.S)


def test_no_load_is_non_coherent():
    files = [f for e in ("cu", "cuh", "h") for f in glob.glob(os.path.join(CSRC, "*." + e))]
    assert any("launch_pdl" in code(f) for f in files)
    found = [(os.path.basename(f), m.group(0)) for f in files for m in re.finditer(r"\b__ldg\b|ld\.global\.nc|\b__restrict(__)?\b", code(f))]
    assert not found, found
