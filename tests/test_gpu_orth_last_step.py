"""Orthogonalised steps whose last result is large: the limit of 8 holds for X between steps only."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_orth import TYPES, exact, make, norm_of

pytestmark = pytest.mark.gpu


def spiked(rows, cols, kind, batch, seed):
    """One element holds nearly all of the norm."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G = 1e-4 * torch.randn(batch, rows, cols, device="cuda", generator=gen)
    G[:, rows // 2, cols // 3] = 1
    return G.to(getattr(torch, TYPES[kind]))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (7, 1), (16, 16), (40, 70), (256, 128), (128, 256), (130, 256), (300, 200)])
@pytest.mark.parametrize("a", [10.0, 1000.0])
def test_one_step_beyond_eight(shape, kind, a):
    """X = a G / |G|. The norm (16 additions of 2^-24, halved by the root), the root, the quotient, the products with it
    and planes of 22 bits stay below 2^-20 together; then the result's rounding, 2^-8 or 2^-24."""
    torch, bl = torch_cuda(), lib()
    G = spiked(*shape, kind, 3, seed=sum(shape))
    got, want = bl.orth(G, steps=1, coefficients=(a, 0.0, 0.0)), exact(G, 1, (a, 0.0, 0.0))
    assert float(want.abs().amax()) > 8
    assert bool(torch.isfinite(got).all())
    far = norm_of(got.double() - want) / norm_of(want)
    assert float(far.amax()) <= 2.0 ** -20 + (2.0 ** -8 if kind == "bf16" else 2.0 ** -24), far


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (40, 70), (130, 256)])
def test_between_steps_it_is_not_finite(shape, kind):
    bl = lib()
    G = spiked(*shape, kind, 2, seed=1)
    got = bl.orth(G, steps=2, coefficients=(10.0, 0.0, 0.0))
    assert bool((~got.isfinite()).any(2).any(1).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_neighbours_of_large_results_are_as_they_are_alone(kind):
    torch, bl = torch_cuda(), lib()
    G = spiked(16, 16, kind, 500, seed=2)
    G[1::2] = make(16, 16, kind, 250, seed=3)
    got = bl.orth(G, steps=1, coefficients=(10.0, 0.0, 0.0))
    assert bool(got.isfinite().all())
    for i in (0, 1, 8, 9, 498, 499):
        assert torch.equal(bl.orth(G[i], steps=1, coefficients=(10.0, 0.0, 0.0)), got[i])
