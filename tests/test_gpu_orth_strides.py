"""Orthogonalised steps of matrices, most of them beyond the small kernel's, whose items lie in each other's gaps or at
distances that are no multiple of a line's: G and results alike, the same bits as for contiguous ones, gaps as they were."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_orth import QUINTIC, TYPES, check

pytestmark = pytest.mark.gpu

# batch, lines, width, distance of the items, of the lines (in values; both multiples of 16 bytes, but for the last)
LAYOUTS = [(3, 300, 160, 160, 480), (3, 300, 160, 168, 504), (2, 200, 304, 304, 608), (4, 150, 264, 264, 8 * 264), (2, 300, 160, 300 * 160 + 8, 160),
           (2, 300, 160, 304 * 160, 160), (2, 300, 160, 300 * 168, 168), (2, 300, 160, 300 * 168 + 16, 168), (4, 1, 400, 400, 400), (4, 1, 400, 408, 400),
           (4, 1, 400, 1200, 400), (3, 2, 600, 600, 1800), (3, 300, 150, 150, 450),
           (2, 3, 400, 1500, 1000), (2, 3, 40, 150, 100), (50, 4, 10, 250, 100), (2, 300, 160, 80 * 320 + 160, 320)]


def view(flat, layout):
    batch, lines, width, item, line = layout
    return flat.as_strided((batch, lines, width), (item, line, 1))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_any_distance_of_items_and_lines(layout, turned, kind):
    torch, bl = torch_cuda(), lib()
    batch, lines, width, item, line = layout
    gen = torch.Generator(device="cuda").manual_seed(item)
    size = (batch - 1) * item + (lines - 1) * line + width
    held = torch.full((size,), 5.0, device="cuda", dtype=getattr(torch, TYPES[kind]))
    G = view(held, layout).copy_(torch.randn(batch, lines, width, device="cuda", generator=gen))
    gaps = torch.ones(size, dtype=torch.bool, device="cuda")
    view(gaps, layout).fill_(False)
    flat = torch.full_like(held, 7.0)
    out = view(flat, layout)
    if turned:
        G, out = G.mT, out.mT
    want = bl.orth(G.mT.contiguous().mT if turned else G.contiguous())
    check(want, G, 5, QUINTIC, kind)
    assert torch.equal(bl.orth(G), want)
    bl.orth(G, out=out)
    assert torch.equal(out, want)
    assert bool((flat[gaps] == 7.0).all()), "a gap was written"
    bl.orth(G, out=G)
    assert torch.equal(G, want) and bool((held[gaps] == 5.0).all())
