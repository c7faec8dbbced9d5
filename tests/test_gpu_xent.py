"""Softmax cross entropy over a vocabulary and its gradients, element by element against the
formulas in 64 bits on the same (bf16 or f32) inputs.

Every tolerance is a bound worked out from the operation's roundings, for the data at hand:
  logits   dim f32 additions: |ds| <= (dim + 8) 2^-23 sum_k |H_rk W_vk|; f32 operands lose another
           2^-22 of that sum to the plane products that are left out
  lse      max |ds| + 2^-20 (1 + |lse|) for exp, log and the joining of tiles; loss: twice that
  P        |dP| <= |g| p expm1(2 max|ds| + 2^-20 (4 + |s| + |lse|)) + u |P|, u = 2^-8 for bf16
           (stored P), 2^-22 for f32
  dH       |dP| |W| + (K + 8) 2^-23 |P||W| + u |dH|; dW likewise
"""
import math

import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu

TYPES = {"f32": "float32", "bf16": "bfloat16"}


def make(rows, dim, vocab, kind, seed=0, pad_h=0, pad_w=0, shift=0, scale=2.0, ignored=0.0):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, TYPES[kind])

    def matrix(r, c, pad, s):
        flat = torch.full((r * (c + pad) + shift,), float("nan"), device="cuda", dtype=dt)
        m = flat[shift:].view(r, c + pad)[:, :c]
        return m.copy_(torch.randn(r, c, device="cuda", generator=gen) * s)
    H, W = matrix(rows, dim, pad_h, scale), matrix(vocab, dim, pad_w, 1 / math.sqrt(dim))
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    if ignored:
        skip = torch.rand(rows, device="cuda", generator=gen) < ignored
        t = torch.where(skip, torch.full_like(t, -100), t)
    g = torch.rand(rows, device="cuda", generator=gen) * 2 - 0.5
    return H, W, t, g


def reference(H, W, t, g, kind):
    """(lse, loss, dH, dW) in f64 and the bounds of their errors, as the module's head says."""
    torch = torch_cuda()
    counted = (t >= 0) & (t < W.shape[0])
    h = torch.where(counted[:, None], H, torch.zeros_like(H)).double()
    w, gd = W.double(), torch.where(counted, g, torch.zeros_like(g)).double()
    at = torch.where(counted, t, torch.zeros_like(t))[:, None]
    rows, dim, vocab = h.shape[0], h.shape[1], w.shape[0]
    s = h @ w.T
    ds = ((dim + 8) * 2.0 ** -23 + (2.0 ** -22 if kind == "f32" else 0)) * (h.abs() @ w.abs().T)
    worst = ds.amax(1)
    lse = torch.logsumexp(s, 1)
    loss = lse - s.gather(1, at)[:, 0]
    e_lse = worst + 2.0 ** -20 * (1 + lse.abs())
    p = (s - lse[:, None]).exp()
    onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
    P = gd[:, None] * (p - onehot)
    u_p = 2.0 ** -8 if kind == "bf16" else 2.0 ** -22
    e_p = gd.abs()[:, None] * p * torch.expm1(2 * worst[:, None] + 2.0 ** -20 * (4 + s.abs() + lse.abs()[:, None]))
    e_p = e_p + u_p * P.abs() + 2.0 ** -22 * gd.abs()[:, None] * onehot
    u_o = 2.0 ** -8 if kind == "bf16" else 2.0 ** -22
    dH, dW = P @ w, P.T @ h
    e_dh = e_p @ w.abs() + (vocab + 8) * 2.0 ** -23 * (P.abs() @ w.abs()) + u_o * dH.abs()
    e_dw = e_p.T @ h.abs() + (rows + 8) * 2.0 ** -23 * (P.abs().T @ h.abs()) + u_o * dW.abs()
    zero = torch.zeros_like(lse)
    return {"lse": (torch.where(counted, lse, zero), e_lse), "loss": (torch.where(counted, loss, zero), 2 * e_lse),
            "dH": (dH, e_dh), "dW": (dW, e_dw)}


def check(got, ref, name):
    torch = torch_cuda()
    value, bound = ref[name]
    assert got.shape == value.shape
    assert bool(torch.isfinite(got).all()), f"{name} is not finite"
    over = ((got.double() - value).abs() - bound - 1e-30).amax().item()
    assert over <= 0, f"{name}: {over:.3e} above its bound (largest bound {bound.amax().item():.3e})"


def run_all(H, W, t, g):
    bl = lib()
    loss, lse = bl.xent(H, W, t)
    dH, dW = bl.xent_grad(H, W, t, lse, g)
    return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


SHAPES = [
    # rows, dim, vocab: one of everything, tile edges on either side, several tiles, ragged
    (1, 1, 1), (1, 8, 2), (1, 64, 1000), (2, 63, 255), (31, 65, 256), (127, 64, 257), (128, 128, 512),
    (129, 257, 513), (300, 320, 1111), (64, 1024, 4100), (513, 72, 3001), (5, 2056, 300),
]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_loss_and_gradients_match_the_formulas(shape, kind):
    H, W, t, g = make(*shape, kind, seed=sum(shape))
    ref, got = reference(H, W, t, g, kind), run_all(H, W, t, g)
    for name in ("lse", "loss", "dH", "dW"):
        check(got[name], ref, name)
    assert got["dH"].dtype == H.dtype and got["dW"].dtype == W.dtype


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [dict(pad_h=3, pad_w=5), dict(pad_h=8, pad_w=8), dict(shift=1), dict(pad_w=1, shift=3)])
def test_strided_and_unaligned_matrices(kind, layout):
    """Rows apart (the gaps hold NaN) and matrices that start off a vector boundary, gradients
    written to matrices of the same layouts without touching their gaps."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(70, 136, 700, kind, seed=3, ignored=0.2, **layout)
    ref = reference(H, W, t, g, kind)
    loss, lse = bl.xent(H, W, t)
    outs = []
    for m in (H, W):
        pad, shift = m.stride(0) - m.shape[1], layout.get("shift", 0)
        flat = torch.full((m.shape[0] * (m.shape[1] + pad) + shift,), 7.0, device="cuda", dtype=m.dtype)
        outs.append((flat, flat[shift:].view(m.shape[0], m.shape[1] + pad)[:, :m.shape[1]]))
    dH, dW = bl.xent_grad(H, W, t, lse, g, dH=outs[0][1], dW=outs[1][1])
    for name, v in (("lse", lse), ("loss", loss), ("dH", dH), ("dW", dW)):
        check(v, ref, name)
    for flat, view in outs:
        view.fill_(7.0)
        assert bool((flat == 7.0).all()), "a gap was written"


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["some", "all", "first", "last", "beyond"])
def test_rows_without_a_target(kind, which):
    """Rows that do not count give zeros, and NaN or infinity in them reaches nothing."""
    torch = torch_cuda()
    H, W, t, g = make(150, 96, 600, kind, seed=5)
    skip = {"some": torch.arange(150, device="cuda") % 3 == 1, "all": torch.ones(150, dtype=torch.bool, device="cuda"),
            "first": torch.arange(150, device="cuda") < 140, "last": torch.arange(150, device="cuda") >= 130,
            "beyond": torch.arange(150, device="cuda") % 2 == 0}[which]
    t[skip] = {"beyond": 600}.get(which, -1)
    H[skip] = float("nan")
    H[skip.nonzero()[0]] = float("inf")
    g[skip] = float("nan")
    ref, got = reference(H, W, t, g, kind), run_all(H, W, t, g)
    for name in ("lse", "loss", "dH", "dW"):
        check(got[name], ref, name)
    assert bool((got["loss"][skip] == 0).all()) and bool((got["lse"][skip] == 0).all())
    assert bool((got["dH"][skip] == 0).all())
    if which == "all":
        assert bool((got["dW"] == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_confident_rows_and_large_logits(kind):
    """Logits of several hundred: the maximum is taken out before the exponential."""
    H, W, t, g = make(64, 64, 900, kind, seed=9, scale=150.0)
    t[:32] = (H[:32].float() @ W.float().T).argmax(1)          # half the rows are sure of their target
    ref, got = reference(H, W, t, g, kind), run_all(H, W, t, g)
    for name in ("lse", "loss", "dH", "dW"):
        check(got[name], ref, name)


@pytest.mark.parametrize("kind,rows,dim,vocab", [("bf16", 70000, 16, 5000), ("f32", 40, 16392, 7000)])
def test_several_pieces_of_the_vocabulary(kind, rows, dim, vocab):
    H, W, t, g = make(rows, dim, vocab, kind, seed=11, ignored=0.1)
    ref, got = reference(H, W, t, g, kind), run_all(H, W, t, g)
    for name in ("lse", "loss", "dH", "dW"):
        check(got[name], ref, name)


def test_one_gradient_alone_is_the_same():
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(200, 128, 900, "bf16", seed=13)
    _, lse = bl.xent(H, W, t)
    dH, dW = bl.xent_grad(H, W, t, lse, g)
    only_h, none_w = bl.xent_grad(H, W, t, lse, g, dW=False)
    none_h, only_w = bl.xent_grad(H, W, t, lse, g, dH=False)
    assert none_w is None and none_h is None
    assert torch.equal(dH, only_h) and torch.equal(dW, only_w)


def test_gradient_against_differences_of_the_loss():
    """d/dx sum g loss along random directions, by central differences of the operator's own loss:
    truncation below h^2 sum |g| (the logits move by at most 1 per unit step), rounding below the
    losses' own error over h."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(20, 40, 150, "f32", seed=17)
    loss, lse = bl.xent(H, W, t)
    dH, dW = bl.xent_grad(H, W, t, lse, g)
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = 2.0 ** -5
    for trial in range(6):
        eh = torch.randn(H.shape, device="cuda", generator=gen) if trial % 2 == 0 else torch.zeros_like(H)
        ew = torch.randn(W.shape, device="cuda", generator=gen) if trial % 2 == 1 else torch.zeros_like(W)
        move = (eh @ W.T + H @ ew.T).abs().amax()
        eh, ew = eh / move, ew / move
        total = [(g.double() * bl.xent(H + s * h * eh, W + s * h * ew, t)[0].double()).sum() for s in (1, -1)]
        measured = (total[0] - total[1]) / (2 * h)
        formula = (dH.double() * eh.double()).sum() + (dW.double() * ew.double()).sum()
        noise = reference(H, W, t, g, "f32")["loss"][1].amax() * g.abs().sum() / h
        assert abs(measured - formula) <= h * h * g.abs().sum() + noise


def test_bits_repeat_and_other_streams_and_graphs():
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(257, 200, 3000, "bf16", seed=19, ignored=0.3)
    first = run_all(H, W, t, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = bl.xent(H, W, t, stream=side)
    dH, dW = bl.xent_grad(H, W, t, lse, g, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for name, v in (("loss", loss), ("lse", lse), ("dH", dH), ("dW", dW)):
        assert torch.equal(first[name], v), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = run_all(H, W, t, g)
    H.copy_(torch.randn_like(H))
    graph.replay()
    torch.cuda.synchronize()
    fresh = run_all(H, W, t, g)
    for name in fresh:
        assert torch.equal(fresh[name], again[name]), name


def test_refusals():
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(8, 16, 32, "bf16")
    _, lse = bl.xent(H, W, t)
    with pytest.raises(TypeError):
        bl.xent(H.half(), W.half(), t)
    with pytest.raises(TypeError):
        bl.xent(H, W.float(), t)
    with pytest.raises(ValueError):
        bl.xent(H, W, t.int())
    with pytest.raises(ValueError):
        bl.xent(H, W, t[:-1])
    with pytest.raises(ValueError):
        bl.xent(H[:, :-1], W, t)
    with pytest.raises(ValueError):
        bl.xent(H.cpu(), W, t)
    with pytest.raises(ValueError):
        bl.xent(H.T.contiguous().T, W, t)
    with pytest.raises(bl.BLError):
        bl.xent(H[:0], W, t[:0])
    with pytest.raises(ValueError):
        bl.xent_grad(H, W, t, lse.double(), g)
    with pytest.raises(ValueError):
        bl.xent_grad(H, W, t, lse, g, dH=torch.empty(8, 15, device="cuda", dtype=H.dtype))
    with pytest.raises(ValueError):
        bl.xent_grad(H, W, t, lse, g, dH=False, dW=False)
    raw = bl.get_lib()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    assert raw.bl_xent(bl.BL_BF16, 8, 16, 32, H.data_ptr(), 16, W.data_ptr(), 16, t.data_ptr(), lse.data_ptr(),
                       lse.data_ptr(), ws.data_ptr(), ws.numel(), None) == 1
    assert b"workspace" in raw.bl_last_error()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 8, 9])
@pytest.mark.parametrize("dim,vocab,pad_w", [(8, 1, 0), (24, 31, 8), (1024, 4099, 0), (1408, 100, 16), (5632, 777, 0), (12000, 300, 0), (6400, 130, 0), (1001, 500, 0)])
def test_loss_of_few_rows(kind, rows, dim, vocab, pad_w):
    """Around the bounds of the kernel for few rows: its most rows, its longest rows, rows of W that
    are no whole vectors, fewer entries than a CTA takes; one row without a target, holding NaN."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(rows, dim, vocab, kind, seed=rows * dim, pad_h=3, pad_w=pad_w)
    if rows > 2:
        t[1] = -5
        H[1] = float("nan")
    ref = reference(H, W, t, g, kind)
    loss, lse = bl.xent(H, W, t)
    check(lse, ref, "lse")
    check(loss, ref, "loss")
    again = bl.xent(H, W, t)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind,rows,dim,vocab,ignored", [
    ("bf16", 1, 64, 300, 0.0), ("bf16", 5, 72, 300, 0.5), ("bf16", 130, 72, 333, 0.9), ("bf16", 300, 129, 1000, 0.4),
    ("f32", 3, 64, 300, 0.3), ("f32", 40, 68, 301, 0.3), ("f32", 200, 131, 700, 0.97), ("f32", 40, 16392, 7000, 0.2)])
def test_nothing_is_read_from_the_workspace_before_it_is_written(kind, rows, dim, vocab, ignored):
    """A workspace of all ones (NaN in every float type) gives the bits that any other gives."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(rows, dim, vocab, kind, seed=23, ignored=ignored)
    want = run_all(H, W, t, g)
    raw, code = bl.get_lib(), bl.BL_F32 if kind == "f32" else bl.BL_BF16
    s = torch.cuda.current_stream().cuda_stream

    def scratch(grad):
        need = raw.bl_xent_workspace(code, rows, dim, vocab, H.data_ptr(), dim, W.data_ptr(), dim, grad)
        return torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ws = scratch(0)
    assert raw.bl_xent(code, rows, dim, vocab, H.data_ptr(), dim, W.data_ptr(), dim, t.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                       ws.data_ptr(), ws.numel() - 256, s) == 0
    assert bool((ws[-256:] == 255).all()), "wrote past the workspace"
    ws = scratch(1)
    dH, dW = torch.full_like(H, float("nan")), torch.full_like(W, float("nan"))
    assert raw.bl_xent_grad(code, rows, dim, vocab, H.data_ptr(), dim, W.data_ptr(), dim, t.data_ptr(), lse.data_ptr(), g.data_ptr(),
                            dH.data_ptr(), dim, dW.data_ptr(), dim, ws.data_ptr(), ws.numel() - 256, s) == 0
    torch.cuda.synchronize()
    assert bool((ws[-256:] == 255).all()), "wrote past the workspace"
    for name, v in (("loss", loss), ("lse", lse), ("dH", dH), ("dW", dW)):
        assert torch.equal(want[name], v), name


@pytest.mark.parametrize("rows", [100, 1000])
def test_equal_weights_round_nothing(rows):
    """Unsure rows of one weight g that lies halfway between two bf16 values: P is -g at the targets
    and g / vocab elsewhere. In units of g that is -(1 - 2^-12), 2^-11 off at most in bf16, so what is
    left is the rounding of dH and dW themselves, uniform within 2^-8: a relative 2-norm of at most
    2^-8 / sqrt(3) + 2^-11 over many values (g itself would be 2^-8 off)."""
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, 512, 4096, "bf16", seed=29)
    W.mul_(2.0 ** -10)
    g = torch.full((rows,), (1 + 2.0 ** -8) * 2.0 ** -10, device="cuda")
    ref = reference(H, W, t, g, "bf16")
    _, lse = bl.xent(H, W, t)
    dH, dW = bl.xent_grad(H, W, t, lse, g)
    for name, v in (("dH", dH), ("dW", dW)):
        off = (v.double() - ref[name][0]).norm() / ref[name][0].norm()
        assert off < 2.0 ** -8 / math.sqrt(3) + 2.0 ** -11, (name, float(off))
