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


def test_lists_that_do_not_overlap_are_taken():
    """Neighbours in one buffer, in any order; inputs that meet one another and are only read; empty tensors
    anywhere; results between inputs."""
    torch, bl = torch_cuda(), lib()
    flat = torch.randn(4000, device="cuda")
    x = list(flat.split([1000, 1, 999, 0, 1500, 500]))
    want = flat * 0.5
    norm = float(flat.double().norm())
    order = [4, 0, 2, 5, 3, 1]
    bl.gclip([x[i] for i in order], norm / 2)
    assert torch.allclose(flat, want, rtol=1e-5)
    source = torch.randn(1000, device="cuda")
    lists = [source, source[100:200], source, source[:0]]
    out = [torch.empty_like(t) for t in lists]
    norm = float(bl.gclip(lists, 1.0, out=out))
    assert abs(norm / float(sum((t.double() ** 2).sum() for t in lists)) ** 0.5 - 1) < 2e-6
    assert all(torch.allclose(o, t / norm, rtol=1e-5) for o, t in zip(out, lists))
    both = torch.randn(8, 100, device="cuda")
    before = both.clone()
    norm = float(bl.gclip(list(both[::2]), 1.0, out=list(both[1::2])))
    assert torch.equal(both[::2], before[::2]) and torch.allclose(both[1::2], before[::2] / norm, rtol=1e-5)


def test_overlaps_are_refused():
    torch, bl = torch_cuda(), lib()
    x = torch.randn(100, device="cuda")
    y = torch.empty_like(x)
    before = x.clone()
    for tensors, out in (([x, x], None), ([x, x[10:20]], None), ([x, y], [y, x]), ([x, y], [x, x]), ([x, x], [x, y])):
        with pytest.raises(bl.BLError):
            bl.gclip(tensors, 0.5, out=out)
    assert torch.equal(x, before)
    assert abs(float(bl.gnorm([x, x])) / (2 * float((x.double() ** 2).sum())) ** 0.5 - 1) < 2e-6
