"""Results that overlap other tensors of a call are refused on the host (no GPU: the addresses are never
looked at)."""
import ctypes
import os

import pytest

BASE = 1 << 30


@pytest.fixture(scope="module")
def bl():
    import matrix_dense_linear_spd_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from matrix_dense_linear_spd_gb300 import build
        build.build()
    return m


def gclip(bl, x, y, sizes, dtype=0):
    n = len(x)
    at = lambda v: (ctypes.c_void_p * n)(*[BASE + k for k in v])
    return bl.get_lib().bl_gclip(n, (ctypes.c_int32 * n)(*[dtype] * n), at(x), at(y), (ctypes.c_int64 * n)(*sizes), 1.0, 4096, 4096,
                                 1 << 30, None)


@pytest.mark.parametrize("x,y,sizes", [
    ([0, 0], [0, 0], [8, 8]),                             # one tensor twice, in place
    ([0, 64, 0], [0, 64, 0], [8, 8, 8]),
    ([0, 16], [0, 16], [8, 8]),                           # views that overlap, in place
    ([64, 0], [64, 0], [4, 32]),
    ([0, 64], [128, 128], [8, 8]),                        # one output twice
    ([0, 64], [128, 156], [8, 8]),
    ([0, 64], [64, 128], [8, 8]),                         # an output that is another tensor's input
    ([0, 64], [64, 0], [8, 8]),                           # each other's
    ([0, 0], [0, 64], [8, 8]),                            # in place, and read again for another output
    ([0, 512], [256, 28], [64, 1]),                       # inside a longer input
    ([0, 8], [512, 16], [64, 1]),
    ([512, 0], [16, 900], [1, 64]),
    ([0], [28], [8]),                                     # its own input, shifted
    ([28], [0], [8]),
])
def test_clip_refuses_overlaps(bl, x, y, sizes):
    assert gclip(bl, x, y, sizes) == 1
    assert b"overlap" in bl.get_lib().bl_last_error()
