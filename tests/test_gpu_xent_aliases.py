"""Results of the cross entropy that overlap other tensors of the call are refused; what lies in the gaps of
another matrix's rows does not overlap it."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradients_that_overlap_are_refused(kind):
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(40, 64, 40, kind, seed=1)
    _, lse = bl.xent(H, W, t)
    kept = [x.clone() for x in (H, W, t, lse, g)]
    other = torch.empty_like(W)
    as_matrix = lambda v: torch.empty(0, dtype=H.dtype, device="cuda").set_(v.untyped_storage(), 0, (1, 1), (1, 1)).expand(1, 1)
    for dH, dW in ((H, None), (None, W), (W, None), (None, H), (other, other), (H[:], False), (False, W[:])):
        with pytest.raises(bl.BLError, match="overlaps"):
            bl.xent_grad(H, W, t, lse, g, dH=dH, dW=dW)
    whole = torch.empty(41, 64, device="cuda", dtype=H.dtype)
    with pytest.raises(bl.BLError, match="overlaps"):
        bl.xent_grad(H, W, t, lse, g, dH=whole[:40], dW=whole[1:])
    one = make(1, 1, 40, kind, seed=1)
    for v in (lse[:1], g[:1], t[:1]):
        with pytest.raises(bl.BLError, match="overlaps"):
            bl.xent_grad(one[0], one[1], t[:1], lse[:1], g[:1], dH=as_matrix(v))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, (H, W, t, lse, g)))


def test_losses_and_workspaces_that_overlap_are_refused():
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(8, 64, 32, "bf16", seed=1)
    raw, s = bl.get_lib(), torch.cuda.current_stream().cuda_stream
    need = raw.bl_xent_workspace(bl.BL_BF16, 8, 64, 32, H.data_ptr(), 64, W.data_ptr(), 64, 0)
    ws = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(8, device="cuda"), torch.empty(8, device="cuda")

    def call(l, e):
        return raw.bl_xent(bl.BL_BF16, 8, 64, 32, H.data_ptr(), 64, W.data_ptr(), 64, t.data_ptr(), l, e, ws.data_ptr(), need, s)
    a, b = loss.data_ptr(), lse.data_ptr()
    for l, e in ((a, a), (a, a + 28), (H.data_ptr(), b), (a, W.data_ptr() + 64), (t.data_ptr() + 32, b), (ws.data_ptr() + 64, b)):
        assert call(l, e) == 1
        assert b"overlaps" in raw.bl_last_error()
    assert call(a, b) == 0
    assert call(a, ws.data_ptr() + (need + 255) // 256 * 256) == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradients_in_the_gaps_are_taken(kind):
    """One buffer holds H and dH side by side, another W, dW and a second W's columns."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(50, 64, 90, kind, seed=3)
    _, lse = bl.xent(H, W, t)
    want = bl.xent_grad(H, W, t, lse, g)
    hh = torch.full((50, 128), 5.0, device="cuda", dtype=H.dtype)
    ww = torch.full((90, 200), 5.0, device="cuda", dtype=H.dtype)
    for h, dh in ((hh[:, :64], hh[:, 64:]), (hh[:, 64:], hh[:, :64])):
        for w, dw in ((ww[:, 8:72], ww[:, 72:136]), (ww[:, 136:], ww[:, :64])):
            h.copy_(H)
            w.copy_(W)
            got = bl.xent_grad(h, w, t, lse, g, dH=dh, dW=dw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(h, H) and torch.equal(w, W)
    # rows of other distances: dH of one buffer's every third row's gap
    buf = torch.full((150, 64), 5.0, device="cuda", dtype=H.dtype)
    buf[::3].copy_(H)
    got = bl.xent_grad(buf[::3], W, t, lse, g, dH=buf[1::3])
    assert torch.equal(got[0], want[0]) and torch.equal(buf[::3], H) and bool((buf[2::3] == 5).all())
