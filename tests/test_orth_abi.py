"""Orthogonalised steps: arguments are checked on the host before any CUDA call (no GPU)."""
import ctypes
import os

import pytest

F = 1 << 24      # addresses that are never looked at: validation fails first


@pytest.fixture(scope="module")
def bl():
    import matrix_dense_linear_spd_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from matrix_dense_linear_spd_gb300 import build
        build.build()
    return m


GOOD = dict(dtype=4, rows=8, cols=300, batch=2, G=F, ldg=8, sg=2400, X=2 * F, ldx=8, sx=2400, steps=5, abc=(3.4445, -4.775, 2.0315), ws=3 * F)
WRONG = [dict(dtype=1), dict(dtype=5), dict(dtype=2), dict(rows=0), dict(rows=(1 << 16) + 1), dict(cols=0), dict(cols=(1 << 16) + 1),
         dict(batch=0), dict(batch=(1 << 20) + 1), dict(rows=1 << 16, cols=1 << 16, batch=1 << 9, ldg=1 << 16, ldx=1 << 16, sx=1 << 32, sg=1 << 32),
         dict(G=None), dict(G=F + 1), dict(ldg=7), dict(sg=-1), dict(X=None), dict(X=F + 1), dict(ldx=7), dict(sx=-128), dict(sx=0), dict(sx=2399),
         dict(ldx=1 << 40), dict(sx=8, ldx=15), dict(steps=0), dict(steps=65), dict(abc=None), dict(abc=(1.0, float("nan"), 0.0)),
         dict(abc=(float("inf"), 1.0, 0.0)), dict(ws=None), dict(ws=3 * F + 128)]


@pytest.mark.parametrize("wrong", WRONG)
def test_orth_refusals(bl, wrong):
    a = dict(GOOD, **wrong)
    abc = (ctypes.c_double * 3)(*a["abc"]) if a["abc"] else None
    assert bl.get_lib().bl_orth(a["dtype"], a["rows"], a["cols"], a["batch"], a["G"], a["ldg"], a["sg"], a["X"], a["ldx"], a["sx"], a["steps"],
                                abc, a["ws"], 1 << 40, None) == 1
    assert bl.get_lib().bl_last_error()


def test_workspace(bl):
    lib = bl.get_lib()
    for bad in ((1, 8, 8, 1), (4, 0, 8, 1), (4, 8, (1 << 16) + 1, 1), (4, 8, 8, 0), (0, 1 << 16, 1 << 16, 1 << 9)):
        assert lib.bl_orth_workspace(*bad) == -1
        assert lib.bl_last_error()


def test_the_tensor_binding_refuses_on_the_host(bl):
    import torch
    x = torch.zeros(4, 8)
    for call in (lambda: bl.orth(3), lambda: bl.orth(x.double()), lambda: bl.orth(x.int())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bl.orth(x), lambda: bl.orth(x[0])):
        with pytest.raises(ValueError):
            call()
