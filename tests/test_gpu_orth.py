"""Orthogonalised steps against the definition in 64 bits.

Tolerances come from the operator's documented roundings, applied to the data at hand in 64 bits (`rounded`): X in
two planes of f16 (22 bits), the products' operands in one (bf16) or two of them, sums that tensor memory cuts by
at most 2^-23.4 of themselves at each of the 16-deep steps of an uncut chain (f32: 24 steps, in chunks). With E the
relative 2-norm by which that differs from the exact result, once with sums cut and once not, the operator's own
result may differ by 2 E (its roundings are others than the emulation's wherever a value lies near a border) and
the rounding of the result, 2^-9 for bf16 as a 2-norm (half of the 2^-8 of the worst element) and 2^-23 for f32."""
import math

import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
TYPES = {"f32": "float32", "bf16": "bfloat16"}


def make(rows, cols, kind, batch=1, seed=0, strong=None, turned=False, pad=0, shift=0):
    """Weak noise, and `strong` strong directions (None: noise only); the gaps of `pad` hold NaN."""
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G = torch.randn(batch, rows, cols, device="cuda", generator=gen)
    if strong:
        G = 0.05 * G + torch.randn(batch, rows, strong, device="cuda", generator=gen) @ torch.randn(batch, strong, cols, device="cuda", generator=gen)
    G = G.to(getattr(torch, TYPES[kind]))
    r, c = (cols, rows) if turned else (rows, cols)
    flat = torch.full((batch * r * (c + pad) + shift,), float("nan"), device="cuda", dtype=G.dtype)
    view = flat[shift:].view(batch, r, c + pad)[:, :, :c]
    if turned:
        view = view.transpose(1, 2)
    return view.copy_(G)


def short_first(X):
    return X.mT if X.shape[-2] > X.shape[-1] else X


def exact(G, steps, abc):
    torch = torch_cuda()
    a, b, c = abc
    X = short_first(G.double())
    norm = torch.linalg.vector_norm(X, dim=(-2, -1), keepdim=True)
    X = X / norm.where(norm > 0, 1.0)
    for _ in range(steps):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT if G.shape[-2] > G.shape[-1] else X


def planes(x, scale):
    torch = torch_cuda()
    hi = (x * scale).half()
    lo = (x * scale - hi.double()).half()
    return hi.double() / scale, lo.double() / scale


def rounded(G, steps, abc, kind, cut):
    """The definition with the operator's roundings, in 64 bits."""
    torch = torch_cuda()
    a, b, c = abc
    X = short_first(G.double())
    norm = torch.linalg.vector_norm(X, dim=(-2, -1), keepdim=True)
    X = X / norm.where(norm > 0, 1.0)

    def product(x, y):
        (xh, xl), (yh, yl) = x, y
        k = xh.shape[-1]
        s = xh @ yh
        if kind == "f32":
            s = s + xh @ yl + xl @ yh
        return s * (1 - cut * 2.0 ** -23.4 * (24 if kind == "f32" else math.ceil(k / 16)))
    turn = lambda p: (p[0].mT, p[1].mT)
    for _ in range(steps):
        x = planes(X, 8192.0)
        A = planes(product(x, turn(x)), 4096.0)
        full = A[0] + A[1] if kind == "f32" else A[0]
        B = planes(b * full + c * product(A, A), 4096.0)
        X = (a * (x[0] + x[1]) + product(B, x)).float().double()
    return X.mT if G.shape[-2] > G.shape[-1] else X


def norm_of(x):
    return x.double().square().sum((-2, -1)).sqrt()


def check(got, G, steps, abc, kind):
    torch = torch_cuda()
    want = exact(G, steps, abc)
    size = norm_of(want)
    off = sum((norm_of(rounded(G, steps, abc, kind, cut) - want) for cut in (0, 1)))
    bound = 2 * off + (2.0 ** -9 if kind == "bf16" else 2.0 ** -23) * size
    assert got.shape == G.shape and got.dtype == G.dtype
    assert bool(torch.isfinite(got).all())
    far = norm_of(got.double() - want)
    assert bool((far <= bound + 1e-300).all()), (far / size, bound / size)


SHAPES = [(1, 1), (1, 5), (7, 1), (1, 3000), (2, 3), (16, 16), (31, 33), (64, 64), (63, 65), (128, 128), (129, 127), (100, 257), (128, 256),
          (130, 256), (127, 300), (257, 100), (300, 300), (256, 512), (517, 1031), (1031, 517), (384, 2000), (2000, 390)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_definition(shape, kind):
    bl = lib()
    for batch, strong, turned in ((1, None, False), (3, 2, False), (2, None, True)):
        G = make(*shape, kind, batch, seed=sum(shape), strong=strong, turned=turned)
        got = bl.orth(G)
        check(got, G, 5, QUINTIC, kind)
        assert got.stride() == G.contiguous().stride() if not turned else got.mT.is_contiguous()
        one = bl.orth(G[0])
        assert bool((one == got[0]).all()), "a matrix depends on what else is in the batch"


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("steps,abc", [(1, QUINTIC), (2, QUINTIC), (9, QUINTIC), (1, CUBIC), (12, CUBIC), (3, (2.0, -1.5, 0.5))])
def test_steps_and_coefficients(steps, abc, kind):
    bl = lib()
    for shape in ((40, 70), (200, 150), (330, 700)):
        G = make(*shape, kind, 2, seed=steps, strong=3)
        check(bl.orth(G, steps=steps, coefficients=abc), G, steps, abc, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(100, 100), (40, 90), (300, 200)])
def test_converges_to_the_nearest_orthogonal_matrix(shape, kind):
    """The cubic's fixed points are singular values of 1: U V^T, to the products' roundings (a relative 2^-11 an
    operand for bf16, 2^-22 for f32, random over the sums; three operands a step and no growth at the end)."""
    torch, bl = torch_cuda(), lib()
    q, _ = torch.linalg.qr(torch.randn(max(shape), min(shape), device="cuda", dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(min(shape), min(shape), device="cuda", dtype=torch.float64))
    s = torch.linspace(0.5, 1.5, min(shape), device="cuda", dtype=torch.float64)
    G = (q * s) @ v.T
    G = (G if shape[0] >= shape[1] else G.T).to(getattr(torch, TYPES[kind]))
    got = bl.orth(G, steps=24, coefficients=CUBIC).double()
    u, _, vh = torch.linalg.svd(G.double(), full_matrices=False)
    far = (got - u @ vh).norm() / math.sqrt(min(shape))
    assert float(far) <= (3 * 2.0 ** -11 + 2.0 ** -9 if kind == "bf16" else 3 * 2.0 ** -22 + 24 * 2.0 ** -23.4)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("exponent", [-120, -70, 0, 60, 120])
def test_any_scale(kind, exponent):
    """The result does not depend on G's scale: powers of two change nothing but what f32 holds of tiny values."""
    torch, bl = torch_cuda(), lib()
    for shape in ((50, 60), (200, 300)):
        G = make(*shape, kind, seed=7)[0]
        scaled = (G.double() * 2.0 ** exponent).to(G.dtype)
        if exponent == -120:
            scaled = scaled.where(G.abs() > 2.0 ** -5, 0)
            G = G.where(G.abs() > 2.0 ** -5, 0)
        check(bl.orth(scaled), scaled, 5, QUINTIC, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(60, 40), (100, 200), (300, 280)])
def test_zeros_infinities_and_nan_stay_in_their_matrix(kind, shape):
    torch, bl = torch_cuda(), lib()
    G = make(*shape, kind, 5, seed=3)
    clean = bl.orth(G)
    G[1] = 0
    G[2, 3, 4] = float("inf")
    G[3, 0, 0] = float("nan")
    got = bl.orth(G)
    assert bool((got[1] == 0).all()) and bool(got[2].isnan().all()) and bool(got[3].isnan().all())
    for i in (0, 4):
        assert torch.equal(got[i], clean[i])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(33, 70), (128, 136), (200, 333), (700, 260)])
@pytest.mark.parametrize("layout", [dict(pad=3), dict(pad=8), dict(shift=1), dict(pad=5, turned=True), dict(shift=3, turned=True)])
def test_strides_offsets_and_given_results(kind, shape, layout):
    """Gaps in G hold NaN; a result with gaps and offsets of its own keeps them; in place is the same."""
    torch, bl = torch_cuda(), lib()
    G = make(*shape, kind, 2, seed=5, **layout)
    got = bl.orth(G)
    check(got, G, 5, QUINTIC, kind)
    turned = layout.get("turned", False)
    r, c = (shape[1], shape[0]) if turned else shape
    flat = torch.full((2 * r * (c + 7) + 5,), 7.0, device="cuda", dtype=G.dtype)
    out = flat[5:].view(2, r, c + 7)[:, :, :c]
    out = out.transpose(1, 2) if turned else out
    version = out._version
    again = bl.orth(G, out=out)
    assert again is out or again.data_ptr() == out.data_ptr()
    assert out._version > version
    assert torch.equal(out, got)
    out.fill_(7.0)
    assert bool((flat == 7.0).all()), "a gap was written"
    bl.orth(G, out=G)
    assert torch.equal(G, got)


def test_interleaved_batches_and_repeated_matrices():
    """Items side by side in each other's gaps, and one matrix seen several times."""
    torch, bl = torch_cuda(), lib()
    base = torch.randn(70, 3, 40, device="cuda")
    G = base.transpose(0, 1)                               # items 40 values apart, lines 120
    want = bl.orth(G.contiguous())
    assert torch.equal(bl.orth(G), want)
    out = torch.zeros_like(base).transpose(0, 1)
    bl.orth(G, out=out)
    assert torch.equal(out, want)
    same = bl.orth(G[:1].expand(4, -1, -1))
    assert all(torch.equal(same[i], want[0]) for i in range(4))


@pytest.mark.parametrize("kind,batch,rows,cols", [("bf16", 2, 200, 300), ("f32", 1, 130, 700), ("f32", 5, 64, 64)])
def test_other_streams_and_graphs(kind, batch, rows, cols):
    torch, bl = torch_cuda(), lib()
    G = make(rows, cols, kind, batch, seed=9)
    first = bl.orth(G)
    assert torch.equal(first, bl.orth(G))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = bl.orth(G, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = bl.orth(G)
    G.copy_(make(rows, cols, kind, batch, seed=10))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, bl.orth(G))


@pytest.mark.parametrize("kind,batch,rows,cols", [("bf16", 3, 100, 70), ("f32", 2, 64, 200), ("bf16", 1, 300, 130), ("f32", 2, 129, 500)])
def test_nothing_is_read_from_the_workspace_before_it_is_written(kind, batch, rows, cols):
    import ctypes
    torch, bl = torch_cuda(), lib()
    G = make(rows, cols, kind, batch, seed=11)
    want = bl.orth(G)
    raw, code = bl.get_lib(), bl.BL_F32 if kind == "f32" else bl.BL_BF16
    need = raw.bl_orth_workspace(code, cols, rows, batch)
    for fill in (255, 0x7c):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        X = torch.full_like(G, float("nan"))
        assert raw.bl_orth(code, cols, rows, batch, G.data_ptr(), cols, rows * cols, X.data_ptr(), cols, rows * cols, 5,
                           (ctypes.c_double * 3)(*QUINTIC), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert bool((ws[need:] == fill).all()), "wrote past the workspace"
        assert torch.equal(X, want)


@pytest.mark.parametrize("kind,rows,cols", [("bf16", 300, 200), ("f32", 150, 260)])
def test_a_product_that_gave_up_is_seen(kind, rows, cols):
    torch, bl = torch_cuda(), lib()
    G = make(rows, cols, kind, 2, seed=13)
    want = bl.orth(G)
    switch = bl.get_lib().bl_debug_xent_gave_up
    switch(1)
    try:
        got = bl.orth(G)
    finally:
        switch(0)
    assert bool(got.isnan().all())
    assert torch.equal(want, bl.orth(G))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("batch,rows,cols,turned", [(400, 16, 16, False), (1001, 5, 40, False), (333, 60, 64, True), (700, 100, 30, False),
                                                    (305, 128, 100, True), (200, 96, 64, False), (160, 256, 33, False)])
def test_many_small_matrices(kind, batch, rows, cols, turned):
    """Several share a CTA: each comes out as it does alone, whatever its neighbours hold."""
    torch, bl = torch_cuda(), lib()
    G = make(rows, cols, kind, batch, seed=batch, strong=2, turned=turned)
    got = bl.orth(G)
    check(got, G, 5, QUINTIC, kind)
    for i in (0, 1, 7, batch // 2, batch - 1):
        assert torch.equal(bl.orth(G[i]), got[i])
    G[1] = float("inf")
    G[4, 0, 0] = float("nan")
    G[5] = 0
    again = bl.orth(G)
    assert bool(again[[1, 4]].isnan().all()) and bool((again[5] == 0).all())
    rest = torch.ones(batch, dtype=torch.bool, device="cuda")
    rest[[1, 4, 5]] = False
    assert torch.equal(again[rest], got[rest])
    # coefficients that diverge: nothing finite, or what the definition gives
    wild = bl.orth(G, steps=20, coefficients=(30.0, 9.0, 1.0))
    assert bool(wild[rest].isnan().any(2).any(1).all()) and bool((wild[5] == 0).all())


def test_symmetric_matrices_stay_symmetric():
    """X of a symmetric G: every product is computed from symmetric operands, A and B are symmetric to the bit."""
    torch, bl = torch_cuda(), lib()
    G = torch.randn(300, 300, device="cuda")
    G = G + G.T
    X = bl.orth(G).double()
    assert float((X - X.T).norm() / X.norm()) < 2.0 ** -18


def test_refusals():
    torch, bl = torch_cuda(), lib()
    G = make(20, 30, "f32")[0]
    for bad in (G.half(), G.double(), 3):
        with pytest.raises(TypeError):
            bl.orth(bad)
    with pytest.raises(ValueError):
        bl.orth(G.cpu())
    with pytest.raises(ValueError):
        bl.orth(G[0])
    with pytest.raises(ValueError):
        bl.orth(G[:, ::2])
    with pytest.raises(ValueError):
        bl.orth(G, coefficients=(1.0, 2.0))
    with pytest.raises(TypeError):
        bl.orth(G, steps=1.5)
    with pytest.raises(ValueError):
        bl.orth(G, out=torch.empty(20, 31, device="cuda"))
    with pytest.raises(ValueError):
        bl.orth(G, out=torch.empty(30, 20, device="cuda").T)
    for bad in (dict(steps=0), dict(steps=65), dict(steps=-1), dict(coefficients=(float("nan"), 0, 0)), dict(coefficients=(1, float("inf"), 0))):
        with pytest.raises(bl.BLError):
            bl.orth(G, **bad)
    with pytest.raises(bl.BLError):
        bl.orth(G[:0])
    with pytest.raises(bl.BLError):
        bl.orth(G, out=torch.empty(1, 30, device="cuda").expand(20, 30))
    with pytest.raises(bl.BLError):
        bl.orth(G.expand(2, 20, 30), out=torch.empty(1, 20, 30, device="cuda").expand(2, 20, 30))
    flat = torch.zeros(2000, device="cuda")
    for shape in ((20, 30), (300, 3)):
        n = shape[0] * shape[1]
        with pytest.raises(bl.BLError, match="overlaps"):
            bl.orth(flat[:n].view(shape), out=flat[1:n + 1].view(shape))
    X = bl.orth(G.requires_grad_())
    assert not X.requires_grad
