"""Clipping where the norm, or the factor, leaves the range of f32."""
import math

import pytest

from _gpu import lib, torch_cuda
from test_gpu_grads import norm64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", [["float32"], ["bfloat16"], ["float32", "float64", "bfloat16"], ["float64"]])
def test_a_norm_beyond_f32_changes_nothing(kinds):
    """The norm is returned in f32. Where it is infinite there, although every value is finite, the factor is 1 as
    for any norm that the caller sees as not finite."""
    torch, bl = torch_cuda(), lib()
    x = [torch.full((1000,), 3e38, device="cuda", dtype=getattr(torch, k)) for k in kinds]
    before = [t.clone() for t in x]
    out = [torch.zeros_like(t) for t in x]
    assert float(bl.gclip(x, 1.0, out=out)) == math.inf
    assert all(torch.equal(a, b) for a, b in zip(out, before))
    assert float(bl.gclip(x, 1.0)) == math.inf
    assert all(torch.equal(a, b) for a, b in zip(x, before))


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("size,limit", [(1e30, 1e-3), (1e30, 1e-8), (1e35, 1e-5), (1e35, 1e-10)])
def test_factors_below_the_range_of_f32(kind, size, limit):
    """c = limit / norm down to 1e-46, below f32's normal range; its products lie within f32's. Two roundings
    of f32, the norm's error and the type's own: u + 3e-6 as elsewhere."""
    torch, bl = torch_cuda(), lib()
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = [(torch.randn(n, device="cuda", generator=gen).double() * size).to(getattr(torch, kind)) for n in (1, 77, 5000)]
    want = norm64(x)
    y = [torch.empty_like(t) for t in x]
    assert abs(float(bl.gclip(x, limit, out=y)) / want - 1) < 2e-6
    u = 2.0 ** -8 if kind == "bfloat16" else 2.0 ** -23
    for a, b in zip(x, y):
        exact = a.double() * (limit / want)
        assert bool(((b.double() - exact).abs() <= (u + 3e-6) * exact.abs() + 2.0 ** -126).all())
    bl.gclip(x, limit)
    assert all(torch.equal(a, b) for a, b in zip(x, y))
