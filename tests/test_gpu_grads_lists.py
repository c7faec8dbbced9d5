"""What the lists of the gradient operators may be: generators, whose tensors nobody else may hold."""
import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu


def test_tensors_of_a_generator_are_held():
    torch, bl = torch_cuda(), lib()
    x = [torch.randn(100, device="cuda") for _ in range(3)]
    want = float(bl.gnorm(x))
    taken = []

    def fresh():
        for t in x:
            y = torch.empty_like(t)
            taken.append((y.data_ptr(), y.data_ptr() + 4 * y.numel()))
            yield y
    norm = bl.gclip(x, 0.5, out=fresh())
    assert all(not lo <= norm.data_ptr() < hi for lo, hi in taken), "the norm lies in an output that was given up"
    assert float(norm) == want
    assert float(bl.gnorm(t.clone() for t in x)) == want
    out = [torch.empty_like(t) for t in x]
    bl.gclip(iter(x), 0.5, out=iter(out))
    assert all(torch.allclose(o, t * (0.5 / want)) for o, t in zip(out, x))


def test_a_list_that_shrinks_while_the_outputs_are_made():
    torch, bl = torch_cuda(), lib()
    x = [torch.randn(100, device="cuda") for _ in range(3)]

    def shrinking():
        while x:
            yield torch.empty_like(x.pop())
    with pytest.raises(ValueError):
        bl.gclip(x, 0.5, out=shrinking())
