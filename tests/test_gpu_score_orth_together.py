"""Scores and orthogonalised steps next to each other: calls at once on several streams, graphs that replay while
other calls run, matrices whose batch decides how they are cut into tiles, the largest counts of rows and alternatives."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_orth import make as matrix
from test_gpu_score import equal, score_all, weights
from test_gpu_xent import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(300, 200), (517, 600), (1100, 300)])
def test_a_matrix_does_not_depend_on_its_batch(kind, rows, cols):
    torch, bl = torch_cuda(), lib()
    G = matrix(rows, cols, kind, 70, seed=1)
    got = bl.orth(G)
    for n in (1, 2, 9):
        assert torch.equal(bl.orth(G[:n]), got[:n]), n


def test_calls_at_once():
    """Four streams: scores with alternatives, gradients, tiled and small matrices; each as it is alone."""
    torch, bl = torch_cuda(), lib()
    a, b = make(300, 200, 20000, "bf16", seed=1), make(5, 300, 9000, "f32", seed=2)
    ga, gb = weights(300), weights(5)
    big, small = matrix(700, 500, "bf16", 3, seed=3), matrix(60, 50, "f32", 300, seed=4)

    def calls():
        return [lambda: score_all(*a[:3], 20, *ga), lambda: score_all(*b[:3], 7, *gb), lambda: {"x": bl.orth(big)}, lambda: {"x": bl.orth(small)}]
    want = [f() for f in calls()]
    streams = [torch.cuda.Stream() for _ in range(4)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for s, f in zip(streams, calls()):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert equal(w, g)


def test_a_graph_replays_beside_eager_calls():
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(200, 64, 30000, "bf16", seed=5)
    G = matrix(400, 300, "f32", 2, seed=6)
    want = score_all(H, W, t, 10), bl.orth(G)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = score_all(H, W, t, 10), bl.orth(G)
    side = torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(side):
            graph.replay()
        now = score_all(H, W, t, 10), bl.orth(G)
    torch.cuda.synchronize()
    for x in (held, now):
        assert equal(want[0], x[0]) and torch.equal(want[1], x[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_as_many_alternatives_as_entries(kind):
    """Every token is an alternative: all of them, in order."""
    torch, bl = torch_cuda(), lib()
    for rows in (1, 7, 40, 300):
        for vocab in (1, 2, 31, 32):
            H, W, t, _ = make(rows, 40, vocab, kind, seed=vocab)
            top_logp, top_id = bl.score(H, W, t, vocab)[3:]
            assert bool((top_id.sort(1).values == torch.arange(vocab, device="cuda")).all())
            assert bool((top_logp[:, :-1] >= top_logp[:, 1:]).all())
            assert float((top_logp.double().exp().sum(1) - 1).abs().max()) < 1e-5


def test_many_rows_of_few_entries():
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(200000, 8, 40, "bf16", seed=8, ignored=0.5)
    out = score_all(H, W, t, 3)
    s = H.double() @ W.double().T
    x = torch.log_softmax(s, 1)
    c = t >= 0
    assert float((out["logp"][c].double() - x[c].gather(1, t[c][:, None])[:, 0]).abs().max()) < 1e-4
    assert float((out["top_logp"][c].double() - x[c].topk(3, 1).values).abs().max()) < 1e-4
    assert bool((out["top_id"][~c] == -1).all()) and bool((out["entropy"][~c] == 0).all())


def test_shared_vectors_and_views():
    """One row of hidden vectors for all tokens (columns of the same memory), H a view into W: reading is shared."""
    torch, bl = torch_cuda(), lib()
    _, W, _, _ = make(1, 64, 500, "f32", seed=9)
    t = torch.arange(100, device="cuda")
    a = score_all(W[100:200], W, t, 4)
    b = score_all(W[100:200].clone(), W, t, 4)
    assert equal(a, b)
    g, e = weights(100)
    dH, dW = bl.score_grad(W[100:200], W, t, a["lse"], a["entropy"], g, e)
    cH, cW = bl.score_grad(W[100:200].clone(), W, t, a["lse"], a["entropy"], g, e)
    assert torch.equal(dH, cH) and torch.equal(dW, cW)
    with pytest.raises(bl.BLError):
        bl.score_grad(W[100:200], W, t, a["lse"], a["entropy"], g, e, dH=W[:100])


def spread(m, ld):
    """m's rows ld values apart, in memory that nobody else needs."""
    torch = torch_cuda()
    flat = torch.empty((m.shape[0] - 1) * ld + m.shape[1], device="cuda", dtype=m.dtype)
    return flat.as_strided(m.shape, (ld, 1)).copy_(m)


@pytest.mark.parametrize("rows,cols", [(100, 200), (2200, 90), (300, 160)])
def test_steps_of_matrices_whose_offsets_pass_32_bits(rows, cols):
    torch, bl = torch_cuda(), lib()
    G = matrix(rows, cols, "bf16", 1, seed=3)[0]
    ld = (5 << 30) // rows // 8 * 8
    far = spread(G, ld)
    want = bl.orth(G)
    assert torch.equal(bl.orth(far), want)
    assert torch.equal(bl.orth(far.T), want.T)
    assert torch.equal(bl.orth(far, out=far), want)


@pytest.mark.parametrize("rows", [1, 60, 200])
def test_scores_of_vectors_whose_offsets_pass_32_bits(rows):
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, 72, 2000, "bf16", seed=4)
    g, e = weights(rows)
    want = score_all(H, W, t, 5, g, e)
    far = spread(W, (5 << 30) // 2000 // 8 * 8)
    assert equal(score_all(H, far, t, 5, g, e), want)
    if rows > 1:
        assert equal(score_all(spread(H, (5 << 30) // rows // 8 * 8), W, t, 5, g, e), want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_small_matrix_that_gave_up_is_seen(kind):
    torch, bl = torch_cuda(), lib()
    G = matrix(60, 40, kind, 200, seed=5)
    want = bl.orth(G)
    switch = bl.get_lib().bl_debug_xent_gave_up
    switch(1)
    try:
        got = bl.orth(G)
    finally:
        switch(0)
    assert bool(got.isnan().all()) and torch.equal(bl.orth(G), want)
