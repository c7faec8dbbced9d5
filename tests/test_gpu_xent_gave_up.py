"""A product that gave up waiting is seen in every result of the call, whichever of them are wanted. Nothing is
made to wait: the flag that such a product raises is set after products that ended well."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import make, run_all

pytestmark = pytest.mark.gpu


@pytest.fixture
def gave_up():
    torch_cuda()
    switch = lib().get_lib().bl_debug_xent_gave_up
    yield lambda: switch(1)
    switch(0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,pad", [(20, 0), (300, 0), (300, 3)])
def test_every_result_says_so(kind, rows, pad, gave_up):
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(rows, 96, 1111, kind, seed=rows, pad_w=pad)
    t[5] = -1
    want = run_all(H, W, t, g)
    buffer = torch.full((1111, 96 + pad), 7.0, device="cuda", dtype=H.dtype)
    dW = buffer[:, :96]
    gave_up()
    loss, lse = bl.xent(H, W, t)
    counts = t >= 0
    assert bool(loss[counts].isnan().all()) and bool(lse[counts].isnan().all())
    for left_out in ({}, {"dH": False}, {"dW": False}):
        dW.fill_(7.0)
        got = bl.xent_grad(H, W, t, want["lse"], g, **{"dW": dW, **left_out})
        for x in got:
            assert x is None or bool(x.isnan().all()), left_out
    assert bool((buffer[:, 96:] == 7).all())
    assert bl.get_lib().bl_debug_xent_gave_up(0) == 0
    again = run_all(H, W, t, g)
    assert all(torch.equal(want[k], again[k]) for k in want)
    only = bl.xent_grad(H, W, t, want["lse"], g, dH=False)[1]
    assert torch.equal(only, want["dW"])
