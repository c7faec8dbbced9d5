"""How close the cross entropy comes where its worst-case bounds say little: rows that are sure of
their target, whose loss and whose P at the target are differences of nearly equal numbers, and the f32
form's three planes and short sums.

u = 2^-24. The matrix instructions cut sums towards zero, by 2 u of a partial sum at most for 16 products,
so a logit is off by ds <= (dim / 16 + 8) 2 u sum_k |H_rk W_vk| (rounded sums of f32 products: less)."""
import math

import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import TYPES, make

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def sure_rows(rows, dim, vocab, kind, level, gap, seed=0):
    """Rows with a target of their own (as far as the vocabulary goes), `gap` above logits that lie around `level`."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, TYPES[kind])
    W = torch.randn(vocab, dim, device="cuda", generator=gen) / math.sqrt(dim)
    # `level` is spread over every 8th column, so that partial sums climb to it along the whole of K
    W[:, ::8] = 1.0
    t = (torch.arange(rows, device="cuda") * 7) % vocab
    H = torch.randn(rows, dim, device="cuda", generator=gen) * 0.25
    own = W[t].clone()
    own[:, ::8] = 0
    H += own * (gap / (own * own).sum(1, keepdim=True))
    H[:, ::8] = level / (dim // 8)
    g = torch.rand(rows, device="cuda", generator=gen) + 0.5
    return H.to(dt), W.to(dt), t, g


def exact(H, W, t):
    h, w, r = H.double(), W.double(), H.shape[0]
    s = h @ w.T
    at = (range(r), t)
    rest = s - s[at][:, None]
    rest[at] = -math.inf
    loss = rest.exp().sum(1).log1p()                                   # lse - s_t, without cancellation
    steps = (H.shape[1] / 16 + 8) * 2 * U
    ds = steps * (h.abs() @ w.abs().T).amax(1)
    return s, loss, ds


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 8, 100, 300])
@pytest.mark.parametrize("level", [0.0, 30.0, 1000.0, -1000.0])
def test_loss_of_sure_rows(kind, rows, level):
    """loss = log(1 + sum of exp of differences of logits): relative error expm1(2 ds) from the logits and
    what f32 leaves of a sum and a logarithm near 1, 4 u absolute and 2^-18 relative. (lse - s_t in f32 would be
    off by u |lse|: 6e-5 at 1000.)"""
    bl = lib()
    H, W, t, g = sure_rows(rows, 64, 500, kind, level, 13.0, seed=rows)
    s, want, ds = exact(H, W, t)
    loss, lse = bl.xent(H, W, t)
    assert float(want.median()) < 1e-2 and bool((loss >= 0).all())
    assert bool(((loss.double() - want).abs() <= want * (2 * ds).expm1() + 2.0 ** -18 * want + 4 * U).all())
    assert bool(((lse.double() - (want + s[range(rows), t])).abs() <= ds + 2 * U * (1 + lse.abs())).all())
