"""Token scores (log probability, entropy, alternatives) and their gradients, element by element against the
formulas in 64 bits on the same (bf16 or f32) inputs.

Every tolerance is a bound worked out from the operation's roundings, for the data at hand, with x = log p:
  logits   ds as in the cross entropy's tests: (dim + 8) 2^-23 sum_k |H_rk W_vk|, f32 operands 2^-22 of it more
  lse      worst + 2^-20 (1 + |lse|), worst = max ds; logp and the alternatives' values: twice that
  entropy  d entropy = -sum p (x + entropy) ds and sum p |x + entropy| <= 2 entropy: 4 worst (entropy + worst);
           its own arithmetic: 2^-20 (1 + entropy), and 2^-22 sum p x^2 from exponentials of a rounded x
  P        with dx = 2 worst + 2^-20 (4 + |s| + |lse|) and q = expm1(dx), the relative error of p:
           |g| p q + |e| p (q |x + entropy| + (1 + q) (dx + d entropy + 2^-22 (|x| + entropy))), the terms' own
           rounding 2^-22 (|g| (p + onehot) + |e| p |x + entropy|), and u |P|, u = 2^-8 (bf16), 2^-22 (f32)
  dH, dW   |dP| |W| + (K + 8) 2^-23 |P| |W| + u |dH|; dW likewise
"""
import math

import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import SHAPES, make

pytestmark = pytest.mark.gpu


def weights(rows, seed=1):
    torch = torch_cuda()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, device="cuda", generator=gen), torch.rand(rows, device="cuda", generator=gen) - 0.3


def reference(H, W, t, kind, g=None, e=None):
    """{name: (value, bound)} in f64, "x" the log probabilities of all tokens."""
    torch = torch_cuda()
    counted = (t >= 0) & (t < W.shape[0])
    h = torch.where(counted[:, None], H, torch.zeros_like(H)).double()
    w = W.double()
    at = torch.where(counted, t, torch.zeros_like(t))[:, None]
    rows, dim, vocab = h.shape[0], h.shape[1], w.shape[0]
    s = h @ w.T
    ds = ((dim + 8) * 2.0 ** -23 + (2.0 ** -22 if kind == "f32" else 0)) * (h.abs() @ w.abs().T)
    worst = ds.amax(1)
    lse = torch.logsumexp(s, 1)
    x = s - lse[:, None]
    p = x.exp()
    entropy = -(p * x.clamp(min=-1e300)).sum(1)
    e_lse = worst + 2.0 ** -20 * (1 + lse.abs())
    e_entropy = 4 * worst * (entropy + worst) + 2.0 ** -20 * (1 + entropy) + 2.0 ** -22 * (p * x.clamp(min=-1e100) ** 2).sum(1)
    zero = torch.zeros_like(lse)
    out = {"x": (x, 2 * e_lse), "lse": (torch.where(counted, lse, zero), e_lse), "logp": (torch.where(counted, x.gather(1, at)[:, 0], zero), 2 * e_lse),
           "entropy": (torch.where(counted, entropy, zero), e_entropy), "counted": counted}
    if g is not None:
        gd = torch.where(counted, g, torch.zeros_like(g)).double()[:, None]
        ed = torch.where(counted, e, torch.zeros_like(e)).double()[:, None]
        onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
        far = (x + entropy[:, None]).abs()
        P = gd * (onehot - p) - ed * p * (x + entropy[:, None])
        dx = 2 * worst[:, None] + 2.0 ** -20 * (4 + s.abs() + lse.abs()[:, None])
        q = torch.expm1(dx)
        u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -22
        e_p = gd.abs() * p * q + ed.abs() * p * (q * far + (1 + q) * (dx + e_entropy[:, None] + 2.0 ** -22 * (x.abs() + entropy[:, None])))
        e_p = e_p + 2.0 ** -22 * (gd.abs() * (p + onehot) + ed.abs() * p * far) + u * P.abs()
        dH, dW = P @ w, P.T @ h
        out["dH"] = (dH, e_p @ w.abs() + (vocab + 8) * 2.0 ** -23 * (P.abs() @ w.abs()) + u * dH.abs())
        out["dW"] = (dW, e_p.T @ h.abs() + (rows + 8) * 2.0 ** -23 * (P.abs().T @ h.abs()) + u * dW.abs())
    return out


def check(got, ref, name):
    torch = torch_cuda()
    value, bound = ref[name]
    assert got.shape == value.shape
    assert bool(torch.isfinite(got).all()), f"{name} is not finite"
    over = ((got.double() - value).abs() - bound - 1e-30).amax().item()
    assert over <= 0, f"{name}: {over:.3e} above its bound (largest bound {bound.amax().item():.3e})"


def check_top(top_logp, top_id, ref, top):
    """The k-th value is the k-th largest to the logits' accuracy, every index is where its value is, no index
    comes twice, and the values fall."""
    torch = torch_cuda()
    x, bound = ref["x"]
    rows = x.shape[0]
    assert top_logp.shape == top_id.shape == (rows, top)
    c = ref["counted"]
    assert bool((top_logp[~c] == 0).all()) and bool((top_id[~c] == -1).all())
    if top == 0 or not bool(c.any()):
        return
    x, bound, v, i = x[c], bound[c][:, None], top_logp[c].double(), top_id[c]
    assert bool(((i >= 0) & (i < x.shape[1])).all())
    assert bool(((v - x.topk(top, 1).values).abs() <= bound).all())
    assert bool(((v - x.gather(1, i)).abs() <= bound).all())
    assert bool((top_logp[c][:, :-1] >= top_logp[c][:, 1:]).all())
    same = top_logp[c][:, :-1] == top_logp[c][:, 1:]
    order = i.sort(1).values
    assert bool((order[:, 1:] != order[:, :-1]).all())
    return same


def score_all(H, W, t, top, g=None, e=None):
    bl = lib()
    names = ("logp", "entropy", "lse", "top_logp", "top_id")
    out = dict(zip(names, bl.score(H, W, t, top)))
    if g is not None:
        out["dH"], out["dW"] = bl.score_grad(H, W, t, out["lse"], out["entropy"], g, e)
    return out


def equal(a, b):
    torch = torch_cuda()
    return all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_and_gradients_match_the_formulas(shape, kind):
    H, W, t, _ = make(*shape, kind, seed=sum(shape))
    g, e = weights(shape[0])
    top = min(shape[2], (0, 1, 5, 20, 32)[sum(shape) % 5])
    ref, got = reference(H, W, t, kind, g, e), score_all(H, W, t, top, g, e)
    for name in ("lse", "logp", "entropy", "dH", "dW"):
        check(got[name], ref, name)
    check_top(got["top_logp"], got["top_id"], ref, top)
    assert got["dH"].dtype == H.dtype and got["dW"].dtype == W.dtype


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1, 3, 20, 32])
@pytest.mark.parametrize("rows,dim,vocab", [(700, 64, 30001), (130, 200, 40000), (2000, 24, 9999), (9, 40, 70001), (128, 64, 50000)])
def test_alternatives_over_many_tiles(rows, dim, vocab, top, kind):
    """More tiles than the device runs at once: the rows' floors rise on the way."""
    H, W, t, _ = make(rows, dim, vocab, kind, seed=rows + top, ignored=0.2)
    ref, got = reference(H, W, t, kind), score_all(H, W, t, top)
    for name in ("lse", "logp", "entropy"):
        check(got[name], ref, name)
    check_top(got["top_logp"], got["top_id"], ref, top)
    assert equal(got, score_all(H, W, t, top))


def rows_of_logits(values, rows, kind):
    """H and W whose logits are `values` (vocab) for every row, exactly."""
    torch = torch_cuda()
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    H = torch.zeros(rows, 8, device="cuda", dtype=dt)
    H[:, 0] = 1
    W = torch.zeros(len(values), 8, device="cuda", dtype=dt)
    W[:, 0] = values.to(dt)
    return H, W


ORDERS = ["rising", "falling", "equal", "steps", "last", "two", "zeros"]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 3000), (3, 9001), (8, 3000), (100, 30000), (300, 30011), (1500, 9001)])
@pytest.mark.parametrize("order", ORDERS)
def test_equal_values_and_any_order(order, rows, vocab, kind):
    """Ties go to the lowest index; values that rise or fall along the whole vocabulary are found."""
    torch = torch_cuda()
    i = torch.arange(vocab, device="cuda")
    values = {"rising": (i * 256 // vocab).float() / 16, "falling": (255 - i * 256 // vocab).float() / 16, "equal": torch.full_like(i, 3).float(),
              "steps": (i % 7).float(), "last": (i >= vocab - 3).float(), "two": (i % 2048 == 2047).float() * 4,
              "zeros": torch.where(i % 2 == 0, -0.0, 0.0)}[order]
    H, W = rows_of_logits(values, rows, kind)
    t = torch.randint(0, vocab, (rows,), device="cuda")
    top = 17
    got = score_all(H, W, t, top)
    exact = values.double()
    want_value, want = torch.sort(exact + 0.0, dim=0, descending=True, stable=True)
    assert bool((got["top_id"] == want[:top]).all()), (got["top_id"][0], want[:top])
    lse = torch.logsumexp(exact, 0)
    assert bool(((got["top_logp"].double() - (want_value[:top] - lse)).abs() <= 2.0 ** -20 * (2 + lse.abs())).all())
    assert bool(((got["logp"].double() - (exact[t] - lse)).abs() <= 2.0 ** -20 * (2 + lse.abs())).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 4, 50, 300])
def test_masked_logits(kind, rows):
    """Minus infinity and the type's lowest value: no share in entropy and gradients, a place behind all others
    among the alternatives."""
    torch, bl = torch_cuda(), lib()
    vocab, top = 5000, 6
    values = torch.full((vocab,), -math.inf, device="cuda")
    values[[7, 2000, 4999]] = torch.tensor([1.0, 3.0, 2.0], device="cuda")
    p = torch.softmax(torch.tensor([1.0, 3.0, 2.0], dtype=torch.float64), 0)
    entropy = float(-(p * p.log()).sum())
    for low in (-math.inf, float(torch.finfo(torch.bfloat16).min)):
        masked = values.clamp(min=low) if math.isfinite(low) else values
        H, W = rows_of_logits(masked, rows, kind)
        H[:, 1:] = 0
        t = torch.full((rows,), 7, device="cuda")
        got = score_all(H, W, t, top)
        assert got["top_id"][0, :3].tolist() == [2000, 4999, 7]
        assert got["top_id"][0, 3:].tolist() == [0, 1, 2]
        assert bool((got["top_id"] == got["top_id"][0]).all())
        assert float((got["entropy"] - entropy).abs().amax()) < 2.0 ** -20 * 2
        assert float((got["logp"] - float(p[0].log())).abs().amax()) < 2.0 ** -20 * 3
        assert bool((got["top_logp"][:, 3:] < -1e37).all())
        # in the gradient the masks' logits are wanted, their vectors are not: W finite, H brings the infinity
        if math.isfinite(low):
            g, e = weights(rows)
            dH, dW = bl.score_grad(H, W, t, got["lse"], got["entropy"], g, e, dH=False)
            x = p.log()
            for k, v in enumerate((7, 2000, 4999)):
                want = g.double() * ((1.0 if v == 7 else 0.0) - float(p[k])) - e.double() * float(p[k] * (x[k] + entropy))
                # H is one-hot: the sum over rows; P is rounded to bf16 (f32: 2^-20), the sum once more
                u = 2.0 ** -7 if kind == "bf16" else 2.0 ** -19
                assert abs(float(dW[v, 0]) - float(want.sum())) <= u * float(want.abs().sum()) + 2.0 ** -20 * float((g.abs() + 2 * e.abs()).sum())
            rest = torch.ones(vocab, dtype=torch.bool, device="cuda")
            rest[[7, 2000, 4999]] = False
            assert bool((dW[rest] == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 5, 200])
@pytest.mark.parametrize("what", ["inf", "nan", "all"])
def test_rows_without_a_distribution(kind, rows, what):
    """An infinite or NaN logit, or minus infinity only: NaN, no indices; other rows are as they were."""
    torch = torch_cuda()
    H, W, t, _ = make(rows, 32, 900, kind, seed=3)
    clean = score_all(H, W, t, 4)
    H[0] = {"inf": 0.0, "nan": float("nan"), "all": 0.0}[what]
    if what == "inf":
        H[0, 0] = math.inf
        W[:, 0] = W[:, 0].abs() + 0.1
        clean = score_all(torch.cat([torch.zeros_like(H[:1]), H[1:]]), W, t, 4)
    if what == "all":
        H[0, 0] = -math.inf
        W[:, 0] = W[:, 0].abs() + 0.1
        clean = score_all(torch.cat([torch.zeros_like(H[:1]), H[1:]]), W, t, 4)
    got = score_all(H, W, t, 4)
    for name in ("logp", "entropy", "lse", "top_logp"):
        assert bool(got[name][0].isnan().all()), name
        assert torch.equal(got[name][1:], clean[name][1:]), name
    assert bool((got["top_id"][0] == -1).all()) and torch.equal(got["top_id"][1:], clean["top_id"][1:])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [dict(pad_h=3, pad_w=5), dict(pad_h=8, pad_w=8), dict(shift=1), dict(pad_w=1, shift=3)])
@pytest.mark.parametrize("rows", [1, 3, 70, 200])
def test_strided_and_unaligned_matrices(kind, layout, rows):
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, 136, 700, kind, seed=3, ignored=0.2 if rows > 3 else 0, **layout)
    g, e = weights(rows)
    ref = reference(H, W, t, kind, g, e)
    got = score_all(H, W, t, 9)
    outs = []
    for m in (H, W):
        pad, shift = max(0, m.stride(0) - m.shape[1]) if m.shape[0] > 1 else 0, layout.get("shift", 0)
        flat = torch.full((m.shape[0] * (m.shape[1] + pad) + shift,), 7.0, device="cuda", dtype=m.dtype)
        outs.append((flat, flat[shift:].view(m.shape[0], m.shape[1] + pad)[:, :m.shape[1]]))
    got["dH"], got["dW"] = bl.score_grad(H, W, t, got["lse"], got["entropy"], g, e, dH=outs[0][1], dW=outs[1][1])
    for name in ("lse", "logp", "entropy", "dH", "dW"):
        check(got[name], ref, name)
    check_top(got["top_logp"], got["top_id"], ref, 9)
    for flat, view in outs:
        view.fill_(7.0)
        assert bool((flat == 7.0).all()), "a gap was written"


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 100, 150])
@pytest.mark.parametrize("which", ["some", "all"])
def test_rows_without_a_target(kind, rows, which):
    torch = torch_cuda()
    H, W, t, _ = make(rows, 96, 600, kind, seed=5)
    g, e = weights(rows)
    skip = torch.arange(rows, device="cuda") % 3 == 1 if which == "some" else torch.ones(rows, dtype=torch.bool, device="cuda")
    t[skip] = 600
    H[skip] = float("nan")
    g[skip] = e[skip] = float("nan")
    ref, got = reference(H, W, t, kind, g, e), score_all(H, W, t, 5, g, e)
    for name in ("lse", "logp", "entropy", "dH", "dW"):
        check(got[name], ref, name)
    check_top(got["top_logp"], got["top_id"], ref, 5)
    for name in ("logp", "entropy", "lse", "top_logp", "dH"):
        assert bool((got[name][skip] == 0).all()), name


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sure_rows_keep_their_digits(kind):
    """Small entropies, log S - T / S, where the logits are exact. -T / S is a sum of one sign over exponentials of
    x of 25 at most, 2^-18 each: within 2^-10 of itself. S is 1 and more, and each addition to the sum that holds
    its 1 rounds by 2^-24 S at most, which log S shows in absolute terms: five additions of a block's pairs, three
    of the part's other blocks and five of the lanes' parts (eight parts), S in (1, 2) for gaps of 8 and more: 13
    times 2^-24 (for gap 2, S = 136, log S of 4.9 is within 2^-10 of itself as well)."""
    torch = torch_cuda()
    for gap in (2.0, 8.0, 16.0, 24.0):
        for rows in (1, 64, 300):
            values = torch.zeros(1000, device="cuda")
            values[123] = gap
            H, W = rows_of_logits(values, rows, kind)
            got = score_all(H, W, torch.full((rows,), 123, device="cuda"), 2)
            x = torch.log_softmax(values.double(), 0)
            p = x.exp()
            rest = float((999 * p[0] * -x[0]) - p[123] * torch.log1p(-999 * p[0]))
            off = float((got["entropy"].double() - rest).abs().amax())
            assert off <= 2.0 ** -10 * rest + 13 * 2.0 ** -24, (gap, off / rest)
            assert bool((got["top_id"] == torch.tensor([123, 0], device="cuda")).all())


@pytest.mark.parametrize("kind,rows,dim,vocab,top", [("bf16", 140000, 16, 9000, 20), ("f32", 40, 16392, 7000, 7), ("bf16", 3, 16393, 20000, 20)])
def test_several_pieces_of_the_vocabulary(kind, rows, dim, vocab, top):
    H, W, t, _ = make(rows, dim, vocab, kind, seed=11, ignored=0.1)
    ref, got = reference(H, W, t, kind), score_all(H, W, t, top)
    for name in ("lse", "logp", "entropy"):
        check(got[name], ref, name)
    check_top(got["top_logp"], got["top_id"], ref, top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradient_without_entropy_is_the_cross_entropys(kind):
    """e = 0: minus the gradient of sum g loss, to the bit."""
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(200, 128, 900, kind, seed=13, ignored=0.2)
    g, _ = weights(200)
    logp, entropy, lse, _, _ = bl.score(H, W, t)
    loss, lse_x = bl.xent(H, W, t)
    dH, dW = bl.score_grad(H, W, t, lse_x, entropy, g, torch.zeros_like(g))
    xH, xW = bl.xent_grad(H, W, t, lse_x, g)
    assert bool((dH == -xH).all()) and bool((dW == -xW).all())
    assert float((logp + loss).abs().amax()) < 2.0 ** -20 * 20


def test_gradient_against_differences():
    """d/dx sum g logp + e entropy along random directions by central differences of the operator's own scores.
    With logits moving by h at most: third derivatives of logp are below 2, of the entropy below 8 (1 + log vocab)."""
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(20, 40, 150, "f32", seed=17)
    g, e = weights(20)
    _, entropy, lse, _, _ = bl.score(H, W, t)
    dH, dW = bl.score_grad(H, W, t, lse, entropy, g, e)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ref = reference(H, W, t, "f32")
    h = 2.0 ** -5
    for trial in range(6):
        eh = torch.randn(H.shape, device="cuda", generator=gen) if trial % 2 == 0 else torch.zeros_like(H)
        ew = torch.randn(W.shape, device="cuda", generator=gen) if trial % 2 == 1 else torch.zeros_like(W)
        move = (eh @ W.T + H @ ew.T).abs().amax()
        eh, ew = eh / move, ew / move
        total = []
        for s in (1, -1):
            logp, ent, _, _, _ = bl.score(H + s * h * eh, W + s * h * ew, t)
            total.append((g.double() * logp.double()).sum() + (e.double() * ent.double()).sum())
        measured = (total[0] - total[1]) / (2 * h)
        formula = (dH.double() * eh.double()).sum() + (dW.double() * ew.double()).sum()
        noise = (ref["logp"][1].amax() * g.abs().sum() + ref["entropy"][1].amax() * e.abs().sum()) / h
        assert abs(measured - formula) <= h * h * (g.abs().sum() + 8 * (1 + math.log(150)) * e.abs().sum()) / 3 + noise


def test_one_gradient_alone_is_the_same():
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(200, 128, 900, "bf16", seed=13)
    g, e = weights(200)
    _, entropy, lse, _, _ = bl.score(H, W, t)
    dH, dW = bl.score_grad(H, W, t, lse, entropy, g, e)
    only_h, none_w = bl.score_grad(H, W, t, lse, entropy, g, e, dW=False)
    none_h, only_w = bl.score_grad(H, W, t, lse, entropy, g, e, dH=False)
    assert none_w is None and none_h is None
    assert torch.equal(dH, only_h) and torch.equal(dW, only_w)


@pytest.mark.parametrize("rows,vocab", [(1, 4000), (257, 30000)])
def test_other_streams_and_graphs(rows, vocab):
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, 200, vocab, "bf16", seed=19, ignored=0.3 if rows > 1 else 0)
    g, e = weights(rows)
    first = score_all(H, W, t, 20, g, e)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = dict(zip(("logp", "entropy", "lse", "top_logp", "top_id"), bl.score(H, W, t, 20, stream=side)))
    again["dH"], again["dW"] = bl.score_grad(H, W, t, again["lse"], again["entropy"], g, e, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = score_all(H, W, t, 20, g, e)
    H.copy_(torch.randn_like(H))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert equal(score_all(H, W, t, 20, g, e), held)


@pytest.mark.parametrize("kind,rows,dim,vocab,top", [
    ("bf16", 1, 64, 300, 20), ("bf16", 5, 72, 300, 3), ("bf16", 130, 72, 333, 32), ("bf16", 300, 64, 30000, 9), ("f32", 3, 64, 300, 5),
    ("f32", 40, 68, 301, 0), ("f32", 40, 16392, 7000, 4), ("bf16", 300, 64, 30000, 0), ("f32", 8, 64, 1025, 32)])
def test_nothing_is_read_from_the_workspace_before_it_is_written(kind, rows, dim, vocab, top):
    """A workspace of all ones (NaN, and the largest keys) gives the bits that any other gives."""
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, dim, vocab, kind, seed=23, ignored=0.3 if rows > 5 else 0)
    g, e = weights(rows)
    want = score_all(H, W, t, top, g, e)
    raw, code = bl.get_lib(), bl.BL_F32 if kind == "f32" else bl.BL_BF16
    s = torch.cuda.current_stream().cuda_stream
    need = raw.bl_score_workspace(code, rows, dim, vocab, top, H.data_ptr(), dim, W.data_ptr(), dim)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = {k: torch.full_like(v, 77) for k, v in want.items()}
    assert raw.bl_score(code, rows, dim, vocab, top, H.data_ptr(), dim, W.data_ptr(), dim, t.data_ptr(),
                        *[got[k].data_ptr() or None for k in ("logp", "entropy", "lse", "top_logp", "top_id")], ws.data_ptr(), need, s) == 0
    assert bool((ws[need:] == 255).all()), "wrote past the workspace"
    need = raw.bl_xent_workspace(code, rows, dim, vocab, H.data_ptr(), dim, W.data_ptr(), dim, 1)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    assert raw.bl_score_grad(code, rows, dim, vocab, H.data_ptr(), dim, W.data_ptr(), dim, t.data_ptr(), got["lse"].data_ptr(),
                             got["entropy"].data_ptr(), g.data_ptr(), e.data_ptr(), got["dH"].data_ptr(), dim, got["dW"].data_ptr(), dim,
                             ws.data_ptr(), need, s) == 0
    torch.cuda.synchronize()
    assert bool((ws[need:] == 255).all()), "wrote past the workspace"
    assert equal(want, got)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [20, 300])
def test_a_product_that_gave_up_is_seen(kind, rows):
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, 96, 1111, kind, seed=rows)
    t[5] = -1
    g, e = weights(rows)
    want = score_all(H, W, t, 3, g, e)
    switch = bl.get_lib().bl_debug_xent_gave_up
    switch(1)
    try:
        got = score_all(H, W, t, 3)
        dH, dW = bl.score_grad(H, W, t, want["lse"], want["entropy"], g, e)
    finally:
        switch(0)
    counts = t >= 0
    for name in ("logp", "entropy", "lse", "top_logp"):
        assert bool(got[name][counts].isnan().all()), name
    assert bool((got["top_id"] == -1).all()) and bool(dH.isnan().all()) and bool(dW.isnan().all())
    assert equal(want, score_all(H, W, t, 3, g, e))


def test_refusals_and_what_autograd_sees():
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(8, 16, 32, "bf16")
    g, e = weights(8)
    logp, entropy, lse, _, _ = bl.score(H.requires_grad_(), W, t, 3)
    assert not logp.requires_grad and not entropy.requires_grad
    H = H.detach()
    for bad in (-1, 33):
        with pytest.raises(bl.BLError):
            bl.score(H, W, t, bad)
    with pytest.raises(bl.BLError):
        bl.score(H, W[:4], t % 4, 5)
    with pytest.raises(TypeError):
        bl.score(H, W, t, 1.5)
    with pytest.raises(TypeError):
        bl.score(H.half(), W.half(), t)
    with pytest.raises(ValueError):
        bl.score(H, W, t[:-1])
    with pytest.raises(ValueError):
        bl.score_grad(H, W, t, lse, entropy.double(), g, e)
    with pytest.raises(ValueError):
        bl.score_grad(H, W, t, lse, entropy, g, e[:-1])
    with pytest.raises(ValueError):
        bl.score_grad(H, W, t, lse, entropy, g, e, dH=False, dW=False)
    with pytest.raises(bl.BLError):
        bl.score_grad(H, W, t, lse, entropy, g, e, dH=H)
    dH = torch.empty_like(H)
    version = dH._version
    bl.score_grad(H, W, t, lse, entropy, g, e, dH=dH)
    assert dH._version == version + 1
