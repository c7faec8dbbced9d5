"""Clipping where the norm leaves the range of f32."""
import math

import pytest

from _gpu import lib, torch_cuda

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
