"""The training operators' arguments are checked on the host before any CUDA call (no GPU)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def bl():
    import matrix_dense_linear_spd_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from matrix_dense_linear_spd_gb300 import build
        build.build()
    return m


F = 4096      # an address that is never looked at: validation fails first


def grads(bl, clip, count=1, dtype=0, x=F, y=2 * F, size=10, limit=1.0, norm=F, ws=F, ws_bytes=1 << 20, lists=True):
    kinds, sizes = (ctypes.c_int32 * 1)(dtype), (ctypes.c_int64 * 1)(size)
    xs, ys = (ctypes.c_void_p * 1)(x), (ctypes.c_void_p * 1)(y)
    if not lists:
        kinds = xs = ys = sizes = None
    lib = bl.get_lib()
    if clip:
        return lib.bl_gclip(count, kinds, xs, ys, sizes, limit, norm, ws, ws_bytes, None)
    return lib.bl_gnorm(count, kinds, xs, sizes, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("wrong", [dict(count=-1), dict(count=1 << 25), dict(dtype=2), dict(dtype=6), dict(x=None), dict(x=F + 2),
                                   dict(size=-1), dict(size=1 << 41), dict(norm=None), dict(norm=F + 1), dict(ws=None),
                                   dict(ws=F + 4), dict(ws_bytes=8), dict(lists=False), dict(dtype=4, x=F + 1)])
def test_grads_refusals(bl, clip, wrong):
    assert grads(bl, clip, **wrong) == 1
    assert bl.get_lib().bl_last_error()


@pytest.mark.parametrize("wrong", [dict(y=None), dict(y=2 * F + 2), dict(limit=-0.5), dict(limit=float("nan")), dict(y=F + 4), dict(y=F - 4)])
def test_clip_refusals(bl, wrong):
    assert grads(bl, True, **wrong) == 1


def test_grads_workspace(bl):
    lib = bl.get_lib()
    assert lib.bl_gnorm_workspace(-1) == -1 and lib.bl_gnorm_workspace(1 << 25) == -1
    assert 0 < lib.bl_gnorm_workspace(0) <= lib.bl_gnorm_workspace(5000)


GOOD = dict(dtype=4, rows=8, dim=16, vocab=32, H=F, ldh=16, W=F, ldw=16, t=F, loss=F, lse=F, g=F, dH=F, lddh=16, dW=F, lddw=16, ws=F)
WRONG = [dict(dtype=1), dict(dtype=5), dict(dtype=9), dict(rows=0), dict(rows=(1 << 22) + 1), dict(dim=0), dict(dim=(1 << 16) + 1),
         dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(H=None), dict(H=F + 1), dict(ldh=15), dict(W=None), dict(ldw=15),
         dict(ldw=1 << 40), dict(t=None), dict(t=F + 4), dict(lse=None), dict(ws=None), dict(ws=F + 128)]


@pytest.mark.parametrize("wrong", WRONG + [dict(loss=None), dict(loss=F + 2)])
def test_xent_refusals(bl, wrong):
    a = dict(GOOD, **wrong)
    assert bl.get_lib().bl_xent(a["dtype"], a["rows"], a["dim"], a["vocab"], a["H"], a["ldh"], a["W"], a["ldw"], a["t"], a["loss"],
                                a["lse"], a["ws"], 1 << 40, None) == 1
    assert bl.get_lib().bl_last_error()


@pytest.mark.parametrize("wrong", WRONG + [dict(g=None), dict(dH=None, dW=None), dict(lddh=15), dict(lddw=3), dict(dW=F + 1)])
def test_xent_grad_refusals(bl, wrong):
    a = dict(GOOD, **wrong)
    assert bl.get_lib().bl_xent_grad(a["dtype"], a["rows"], a["dim"], a["vocab"], a["H"], a["ldh"], a["W"], a["ldw"], a["t"], a["lse"],
                                     a["g"], a["dH"], a["lddh"], a["dW"], a["lddw"], a["ws"], 1 << 40, None) == 1


def test_matrix_ops_refuse_the_training_types(bl):
    lib = bl.get_lib()
    for dtype in (bl.BL_BF16, bl.BL_F16):
        assert lib.bl_potrf(0, dtype, 4, 1, F, 4, 16, F, None) == 1
    assert lib.bl_xent_workspace(1, 8, 16, 32, F, 16, F, 16, 0) == -1


def test_the_tensor_binding_refuses_on_the_host(bl):
    """Wrong types and CPU tensors raise before anything is allocated on a GPU."""
    import torch
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: bl.gnorm(3), lambda: bl.gnorm([1]), lambda: bl.gnorm([x.int()]), lambda: bl.gclip([x], "1"),
                 lambda: bl.xent(x.double(), x.double(), t), lambda: bl.xent(x, None, t)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bl.gnorm([x]), lambda: bl.gclip([x], 1.0), lambda: bl.xent(x, x, t),
                 lambda: bl.xent_grad(x, x, t, x[0], x[0])):
        with pytest.raises(ValueError):
            call()
