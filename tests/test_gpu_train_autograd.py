"""The training operators beside autograd: they record nothing, and what they write to counts as changed."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import make

pytestmark = pytest.mark.gpu


def test_what_is_written_counts_as_changed():
    torch, bl = torch_cuda(), lib()
    x = [torch.randn(100, device="cuda"), torch.randn(0, device="cuda")]
    out = [torch.empty_like(t) for t in x]
    before = [t._version for t in x + out]
    bl.gclip(x, 0.5, out=out)
    assert [t._version for t in x] == before[:2] and out[0]._version == before[2] + 1
    bl.gnorm(x)
    assert x[0]._version == before[0]
    bl.gclip(x, 0.5)
    assert x[0]._version == before[0] + 1
    w = torch.randn(100, device="cuda", requires_grad=True)
    y = (w * x[0]).sum()                                # keeps x[0] for w's gradient
    bl.gclip([x[0]], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    H, W, t, g = make(20, 16, 40, "bf16")
    _, lse = bl.xent(H, W, t)
    dH, dW = torch.empty_like(H), torch.empty_like(W)
    bl.xent_grad(H, W, t, lse, g, dH=dH, dW=dW)
    assert dH._version == dW._version == 1 and H._version == make(20, 16, 40, "bf16")[0]._version
    with torch.inference_mode():
        z = torch.ones(10, device="cuda")
    bl.gclip([z], 1.0)                                  # an inference tensor has no counter
    assert abs(float(z.norm()) - 1) < 1e-5


def test_nothing_is_recorded_and_gradients_are_handed_on():
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(50, 32, 300, "f32", seed=2)
    base = torch.randn(50, 32, device="cuda", requires_grad=True)
    h, w = base * 2, W.clone().requires_grad_()
    loss, lse = bl.xent(h, w, t)
    assert not loss.requires_grad and not lse.requires_grad and not bl.gnorm([w]).requires_grad
    dH, dW = bl.xent_grad(h, w, t, lse, g)
    assert not dH.requires_grad and not dW.requires_grad
    h.backward(dH)
    want = base.detach().clone().requires_grad_()
    wd = W.clone().requires_grad_()
    per_row = torch.nn.functional.cross_entropy((want.double() * 2) @ wd.double().T, t, reduction="none")
    (per_row * g.double()).sum().backward()
    # f32 results against 64 bits: relative 2-norms
    assert float((base.grad - want.grad).norm() / want.grad.norm()) < 1e-5
    assert float((dW - wd.grad).norm() / wd.grad.norm()) < 1e-5
    assert "no autograd graph" in bl.xent.__doc__
