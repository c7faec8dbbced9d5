"""Orthogonalised steps: which distances of items and lines of X are refused, against a count of every element (no GPU: a call
that is not refused ends where it wants a device, with status 3)."""
import ctypes
import os
import random

import pytest

F = 1 << 24      # addresses that are never looked at


@pytest.fixture(scope="module")
def bl():
    import matrix_dense_linear_spd_gb300 as m
    import torch
    if torch.cuda.is_available():
        pytest.skip("with a device the calls would run")
    if not os.path.exists(m.LIB_PATH):
        from matrix_dense_linear_spd_gb300 import build
        build.build()
    return m


def call(bl, rows, cols, batch, ldx, sx):
    return bl.get_lib().bl_orth(4, rows, cols, batch, F, rows, rows * cols, 4 * F, ldx, sx, 5, (ctypes.c_double * 3)(1.5, -0.5, 0.0), 16 * F, 1 << 40, None)


def shared(rows, cols, batch, ldx, sx):
    at = [b * sx + c * ldx + r for b in range(batch) for c in range(cols) for r in range(rows)]
    return len(set(at)) < len(at)


LAYOUTS = [(100, 3, 2, 1000, 1200), (100, 3, 2, 1000, 1950), (100, 3, 2, 1000, 950), (100, 3, 2, 1000, 900), (100, 1, 3, 0, 100), (100, 1, 3, 0, 99),
           (10, 4, 100, 100, 250), (10, 5, 7, 70, 10), (10, 5, 8, 70, 10), (8, 300, 2, 8, 2399), (8, 300, 2, 8, 2400), (1, 1, 3, 1, 0), (1, 7, 3, 1, 7)]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_items_that_share_memory_are_refused_and_no_others(bl, layout):
    assert call(bl, *layout) == (1 if shared(*layout) else 3)
    if shared(*layout):
        assert b"overlap" in bl.get_lib().bl_last_error()


def test_any_layout(bl):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(3000):
        rows, cols, batch = rng.randrange(1, 9), rng.randrange(1, 7), rng.randrange(1, 7)
        ldx, sx = rng.randrange(rows, 60), rng.randrange(0, 90)
        s = shared(rows, cols, batch, rows if cols == 1 else ldx, sx)
        seen[s] += 1
        assert call(bl, rows, cols, batch, ldx, sx) == (1 if s else 3), (rows, cols, batch, ldx, sx)
    assert min(seen) > 500
