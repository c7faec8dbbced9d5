"""Token scores: arguments are checked on the host before any CUDA call (no GPU)."""
import ctypes
import os

import pytest

F = 1 << 20      # addresses that are never looked at: validation fails first


@pytest.fixture(scope="module")
def bl():
    import matrix_dense_linear_spd_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from matrix_dense_linear_spd_gb300 import build
        build.build()
    return m


GOOD = dict(dtype=4, rows=8, dim=16, vocab=64, top=3, H=F, ldh=16, W=2 * F, ldw=16, t=3 * F, logp=4 * F, entropy=5 * F, lse=6 * F, top_logp=7 * F,
            top_id=8 * F, g=9 * F, e=10 * F, dH=11 * F, lddh=16, dW=12 * F, lddw=16, ws=13 * F)
WRONG = [dict(dtype=1), dict(dtype=5), dict(dtype=9), dict(rows=0), dict(rows=(1 << 22) + 1), dict(dim=0), dict(dim=(1 << 16) + 1),
         dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(H=None), dict(H=F + 1), dict(ldh=15), dict(W=None), dict(ldw=15),
         dict(ldw=1 << 40), dict(t=None), dict(t=F + 4), dict(lse=None), dict(entropy=None), dict(entropy=F + 2), dict(ws=None), dict(ws=F + 128)]


def score(bl, a):
    return bl.get_lib().bl_score(a["dtype"], a["rows"], a["dim"], a["vocab"], a["top"], a["H"], a["ldh"], a["W"], a["ldw"], a["t"], a["logp"],
                                 a["entropy"], a["lse"], a["top_logp"], a["top_id"], a["ws"], 1 << 40, None)


def grad(bl, a):
    return bl.get_lib().bl_score_grad(a["dtype"], a["rows"], a["dim"], a["vocab"], a["H"], a["ldh"], a["W"], a["ldw"], a["t"], a["lse"],
                                      a["entropy"], a["g"], a["e"], a["dH"], a["lddh"], a["dW"], a["lddw"], a["ws"], 1 << 40, None)


@pytest.mark.parametrize("wrong", WRONG + [dict(top=-1), dict(top=33), dict(top=17, vocab=16), dict(logp=None), dict(top_logp=None),
                                           dict(top_id=None), dict(top_id=F + 4)])
def test_score_refusals(bl, wrong):
    assert score(bl, dict(GOOD, **wrong)) == 1
    assert bl.get_lib().bl_last_error()


@pytest.mark.parametrize("wrong", WRONG + [dict(g=None), dict(e=None), dict(e=F + 1), dict(dH=None, dW=None), dict(lddh=15), dict(lddw=3),
                                           dict(dW=F + 1)])
def test_score_grad_refusals(bl, wrong):
    assert grad(bl, dict(GOOD, **wrong)) == 1
    assert bl.get_lib().bl_last_error()


def test_workspace(bl):
    lib = bl.get_lib()
    for bad in (dict(top=-1), dict(top=33), dict(top=17, vocab=16), dict(dtype=1), dict(rows=0)):
        a = dict(GOOD, **bad)
        assert lib.bl_score_workspace(a["dtype"], a["rows"], a["dim"], a["vocab"], a["top"], F, 16, F, 16) == -1


def test_the_tensor_binding_refuses_on_the_host(bl):
    """Wrong types and CPU tensors raise before anything is allocated on a GPU."""
    import torch
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: bl.score(x.double(), x.double(), t), lambda: bl.score(x, None, t)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bl.score(x, x, t), lambda: bl.score_grad(x, x, t, x[0], x[0], x[0], x[0])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("same", [("logp", "entropy"), ("lse", "logp"), ("top_logp", "lse"), ("top_id", "top_logp"), ("logp", "t"),
                                  ("entropy", "H"), ("top_id", "W"), ("ws", "top_id"), ("ws", "H")])
def test_overlaps_need_a_device_to_be_refused(bl, same):
    """Without a device the call ends before it is enqueued; with one it is refused. Either way it is an error."""
    a = dict(GOOD)
    a[same[0]] = a[same[1]]
    assert score(bl, a) in (1, 3)
