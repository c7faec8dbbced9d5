"""Global gradient norm and clipping against 64-bit sums.

Tolerances: squares are added in f32 over at most 32 values and then in f64, and the norm is
rounded to f32, so its relative error is below (32 + 2) 2^-24 / 2 + 2^-24 < 2e-6 (f64 tensors: the
rounding alone). A scaled value carries that error of the factor, two f32 roundings and its own
type's: relative u + 3e-6 with u = 2^-24, 2^-9, 2^-12 rounded up to whole ulps (f16 results below
2^-14 are spaced 2^-24)."""
import math

import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu

U = {"float32": 2.0 ** -23, "float64": 2.0 ** -50, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -10}


def norm64(tensors):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in tensors))


def check_scaled(x, y, c):
    kind = str(x.dtype).split(".")[1]
    want = x.double() * c
    tol = (U[kind] + 3e-6) * want.abs() + (2.0 ** -24 if kind == "float16" else 0)
    assert bool(((y.double() - want).abs() <= tol).all()), kind


def lists(kind, seed=0):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kinds = ["float32", "bfloat16", "float16", "float64"] if kind == "mixed" else [kind]
    sizes = [1, 2, 3, 7, 8, 0, 31, 255, 256, 1000, 4097, 65536, 100003]
    return [(torch.randn(n, device="cuda", generator=gen) * 0.1).to(getattr(torch, kinds[i % len(kinds)]))
            for i, n in enumerate(sizes)]


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16", "float64", "mixed"])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6, math.inf])
def test_norm_and_clip(kind, max_norm):
    torch, bl = torch_cuda(), lib()
    x = lists(kind)
    want = norm64(x)
    assert abs(float(bl.gnorm(x)) / want - 1) < 2e-6
    c = min(1.0, max_norm / want)
    y = [torch.full_like(t, 9) for t in x]
    norm = bl.gclip(x, max_norm, out=y)
    assert norm.dtype == torch.float32 and abs(float(norm) / want - 1) < 2e-6
    for a, b in zip(x, y):
        check_scaled(a, b, c)
        if c == 1.0:
            assert torch.equal(a, b)
    before = [t.clone() for t in x]
    bl.gclip(x, max_norm)                                  # in place: the same bits
    for a, b in zip(x, y):
        assert torch.equal(a, b)
    if max_norm < want and max_norm > 0:
        assert abs(norm64(x) / max_norm - 1) < 2e-3        # bf16's rounding of what was scaled
    del before


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("shift_x,shift_y", [(0, 0), (1, 1), (3, 0), (0, 5), (2, 7)])
def test_pieces_of_flat_buffers(kind, shift_x, shift_y):
    """Tensors that start anywhere, results that start elsewhere; what lies between is not touched."""
    torch, bl = torch_cuda(), lib()
    dt = getattr(torch, kind)
    counts = [5, 1, 20000, 13, 8191, 8193, 64, 3]
    fx = torch.full((sum(counts) + 20 * len(counts),), float("nan"), device="cuda").to(dt)
    fy = torch.full((fx.numel() + 16,), 7.0, device="cuda").to(dt)
    x, y, at = [], [], 0
    for n in counts:
        x.append(fx[at + shift_x:at + shift_x + n])
        y.append(fy[at + shift_y:at + shift_y + n])
        x[-1].copy_(torch.randn(n, device="cuda"))
        at += n + 20
    want = norm64(x)
    norm = bl.gclip(x, 1.0, out=y)
    assert abs(float(norm) / want - 1) < 2e-6
    for a, b in zip(x, y):
        check_scaled(a, b, 1.0 / want)
        b.fill_(7.0)
    assert bool((fy == 7.0).all())


@pytest.mark.parametrize("count", [1, 64, 65, 999, 1000, 1001, 2500])
def test_many_tensors(count):
    torch, bl = torch_cuda(), lib()
    x = [torch.randn(i % 41, device="cuda") for i in range(count - 1)] + [torch.randn(5000, device="cuda")]
    want = norm64(x)
    y = [torch.empty_like(t) for t in x]
    assert abs(float(bl.gnorm(x)) / want - 1) < 2e-6
    assert abs(float(bl.gclip(x, 0.25 * want, out=y)) / want - 1) < 2e-6
    for a, b in zip(x, y):
        check_scaled(a, b, 0.25)


def test_empty_lists_and_zeros():
    torch, bl = torch_cuda(), lib()
    assert float(bl.gnorm([])) == 0.0 and float(bl.gclip([], 1.0)) == 0.0
    e = [torch.empty(0, device="cuda"), torch.empty(0, 4, device="cuda")]
    assert float(bl.gnorm(e)) == 0.0 and float(bl.gclip(e, 1.0)) == 0.0
    z = [torch.zeros(100, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.bfloat16)]
    for limit in (0.0, 1.0):
        assert float(bl.gclip(z, limit)) == 0.0
        assert all(bool((t == 0).all()) for t in z)


@pytest.mark.parametrize("kind,scale", [("float32", 1e30), ("float32", 1e-30), ("bfloat16", 1e32), ("bfloat16", 1e-35), ("float32", 1e-42)])
def test_squares_beyond_the_range_of_f32(kind, scale):
    torch, bl = torch_cuda(), lib()
    x = [(torch.randn(5000, device="cuda").double() * scale).to(getattr(torch, kind)) for _ in range(3)]
    want = norm64(x)
    rel = 2e-6 if want > 1e-37 else 1e-3                    # the f32 norm itself is subnormal there
    assert abs(float(bl.gnorm(x)) / want - 1) < rel


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_norm_that_is_not_finite_changes_nothing(bad):
    torch, bl = torch_cuda(), lib()
    x = [torch.randn(1000, device="cuda"), torch.randn(77, device="cuda", dtype=torch.float16)]
    x[0][500] = bad
    before = [t.clone() for t in x]
    norm = float(bl.gclip(x, 1.0))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    for a, b in zip(x, before):
        assert torch.equal(a.nan_to_num(nan=123.0), b.nan_to_num(nan=123.0))


def test_memory_orders_streams_graphs_and_repetition():
    torch, bl = torch_cuda(), lib()
    m = bl.colmajor(torch.randn(7, 33, 65, device="cuda"))
    x = [m, torch.randn(8, 5, 6, device="cuda").permute(2, 0, 1), torch.randn(100000, device="cuda")]
    want = norm64(x)
    out = [torch.empty_like(t, memory_format=torch.preserve_format) for t in x]
    first = bl.gclip(x, 1.0, out=out)
    for a, b in zip(x, out):
        check_scaled(a, b, 1.0 / want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = bl.gnorm(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = bl.gclip(x, 1.0, out=out)
    x[2].mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, bl.gnorm(x))


def test_refusals():
    torch, bl = torch_cuda(), lib()
    x = torch.randn(64, device="cuda")
    with pytest.raises(TypeError):
        bl.gnorm([x.to(torch.int32)])
    with pytest.raises(TypeError):
        bl.gnorm([x.to(torch.complex64)])
    with pytest.raises(ValueError):
        bl.gnorm([x, x.cpu()])
    with pytest.raises(ValueError):
        bl.gnorm([x[::2]])
    with pytest.raises(ValueError):
        bl.gnorm([x[:1].expand(64)])
    with pytest.raises(ValueError):
        bl.gclip([x], 1.0, out=[])
    with pytest.raises(ValueError):
        bl.gclip([x], 1.0, out=[x.half()])
    with pytest.raises(ValueError):
        bl.gclip([x.view(8, 8)], 1.0, out=[torch.empty(8, 8, device="cuda").T])
    for limit in (-1.0, math.nan):
        with pytest.raises(bl.BLError):
            bl.gclip([x], limit)
    with pytest.raises(bl.BLError):
        bl.gclip([x[:60]], 1.0, out=[x[4:]])               # the result overlaps its input
