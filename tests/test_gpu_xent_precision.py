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


@pytest.mark.parametrize("kind,rows,dim,level", [("bf16", 1, 4096, 20.0), ("bf16", 100, 4096, 40.0), ("bf16", 300, 4096, 40.0),
                                                 ("bf16", 300, 16384, 40.0), ("f32", 1, 4096, 40.0), ("f32", 100, 4096, 40.0),
                                                 ("f32", 300, 4096, 40.0)])
def test_gradient_of_sure_rows(kind, rows, dim, level):
    """P at the target is g (p - 1), p within 1e-2 of 1. Loss and gradient form the same logits, so ds moves p - 1 by
    (1 - p) expm1(2 ds) only; what is left of s - lse is lse's rounding, d = u |lse| + 2^-21, and, where
    the loss of few rows has been summed by another kernel, both kernels' sums: 16 u sum |HW| at most. Elsewhere |dP| <= g p
    expm1(2 ds + d). Then P's own rounding, dW's sum and dW's rounding."""
    torch, bl = torch_cuda(), lib()
    vocab = 2000
    H, W, t, g = sure_rows(rows, dim, vocab, kind, level, 17.0, seed=dim + rows)
    s, loss, ds = exact(H, W, t)
    assert 1e-6 < float(loss.median()) < 1e-2
    h, w, gd, at = H.double(), W.double(), g.double(), (range(rows), t)
    lse_exact = s[at] + loss
    d = U * lse_exact.abs() + 2.0 ** -21
    if rows <= 8:
        d = d + 16 * U * (h.abs() @ w.abs().T).amax(1)
    p = (s - lse_exact[:, None]).exp()
    P, e_p = p.clone(), p * (2 * ds + d)[:, None].expm1()
    P[at] = (-loss).expm1()
    e_p[at] = -P[at] * (2 * ds).expm1() + d
    P, e_p = P * gd[:, None], e_p * gd[:, None]
    u_p = 2.0 ** -8 if kind == "bf16" else 2.0 ** -20
    e_p = e_p + u_p * P.abs()
    want = P.T @ h
    bound = e_p.T @ h.abs() + (rows + 8) * 2 * U * (P.abs().T @ h.abs()) + u_p * want.abs()
    _, lse = bl.xent(H, W, t)
    dH, dW = bl.xent_grad(H, W, t, lse, g)
    over = (dW.double() - want).abs() - bound
    worst = (dW.double() - want)[t].norm() / want[t].norm()
    assert float(over.amax()) <= 0, f"targets' rows of dW are {float(worst):.2e} off"


@pytest.mark.parametrize("rows", [1 << 17, 1 << 21])
def test_dW_of_many_rows_is_not_biased(rows):
    """Logits of zero: every p is 1 / 300, P is its rounding to bf16, and an entry that is nobody's target gets the sum of as
    many equal terms as there are rows. Cut towards zero in one chain, 2^21 rows would lose 2^-25 a step of
    16, 2^-8 of the sum; chains of 65536 at most lose 2^-13, which leaves dW's own rounding of 2^-9."""
    torch, bl = torch_cuda(), lib()
    H = torch.full((rows, 8), 1 + 2.0 ** -7, device="cuda", dtype=torch.bfloat16)
    W = torch.zeros(300, 8, device="cuda", dtype=torch.bfloat16)
    t, g = torch.zeros(rows, dtype=torch.int64, device="cuda"), torch.ones(rows, device="cuda")
    _, lse = bl.xent(H, W, t)
    _, dW = bl.xent_grad(H, W, t, lse, g, dH=False)
    p = float(torch.tensor(1 / 300).bfloat16())
    want = rows * p * (1 + 2.0 ** -7)
    assert float((dW[1:].double() / want - 1).abs().amax()) <= 2.0 ** -9 + 2.0 ** -12


@pytest.mark.parametrize("rows,vocab", [(64, 3000), (1024, 4000)])
def test_f32_products_are_f32(rows, vocab):
    """Single CTAs and pairs, f32. Three planes and sums cut every 128 of K leave a relative error of about 4e-7 in the
    2-norm, of which f32's own rounding is 1e-7; two planes (2^-17 an element) or uncut sums (1e-5 at K = 32000, 1e-6
    at 4000) would not stay below 1e-6. A vocabulary of one entry shows the logits: lse = s."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(rows, 1024, vocab, "f32", seed=rows, scale=1.0)
    g = g.abs() + 0.5
    for v in (0, 7):
        _, s = bl.xent(H, W[v:v + 1], torch.zeros_like(t))
        want = H.double() @ W[v].double()
        assert float((s.double() - want).norm() / want.norm()) < 1e-6
    _, lse = bl.xent(H, W, t)
    dH, dW = bl.xent_grad(H, W, t, lse, g)
    P = torch.softmax(H.double() @ W.double().T, 1)
    P[range(rows), t] -= 1
    P *= g.double()[:, None]
    for name, got, want in (("dH", dH, P @ W.double()), ("dW", dW, P.T @ H.double())):
        off = float((got.double() - want).norm() / want.norm())
        assert off < 1e-6, (name, off)


@pytest.mark.parametrize("rows", [1, 2, 5, 32])
def test_gradients_of_few_rows_are_rounded_once(rows):
    """P of one row, or of few, scales whole rows of the results: rounded to 8 bits it would put up to 2^-8 on top of
    the results' own rounding. That is uniform within 2^-8 of a value, or less: a relative 2-norm of 2^-8 / sqrt(3) over many
    values, whose mantissas are not all 1; 2^-11 is left for everything else."""
    torch, bl = torch_cuda(), lib()
    for seed in range(24):
        H, W, t, g = make(rows, 512, 2000, "bf16", seed=100 * rows + seed)
        H.add_(W[t] * torch.linspace(0, 10, rows + 24, device="cuda")[seed:seed + rows, None])           # some rows are sure, most are not
        _, lse = bl.xent(H, W, t)
        dH, dW = bl.xent_grad(H, W, t, lse, g)
        P = torch.softmax(H.double() @ W.double().T, 1)
        P[range(rows), t] -= 1
        P *= g.double()[:, None]
        for name, got, want in (("dH", dH, P @ W.double()), ("dW", dW, P.T @ H.double())):
            off = float((got.double() - want).norm() / want.norm())
            assert off < 2.0 ** -8 / math.sqrt(3) + 2.0 ** -11, (name, seed, off)
