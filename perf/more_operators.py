"""More training operators' cases: log probabilities of given tokens with their entropy and the likeliest
alternatives, the gradients of both (a policy's training step), and the orthogonalised step of a weight.

`own = False` computes the plain form in elementary torch operations; `own = True` calls the
package. Sizes are generic: token counts from one to a few thousand, vocabularies of a few
thousand to 131,072 entries, weights from 16 x 16 blocks to 8192 x 4096.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # a token that is being generated, with the alternatives that a serving interface reports: latency
        score_case("score-1", "score", "bf16", 1, 1024, 32000, 20),
        # everything odd, in f32: rows, dim and vocab are no multiples of anything, rows strided
        score_case("score-f32-odd", "score", "f32", 77, 259, 5003, 5, pad=5),
        # an evaluation with the prompts' rows left out: was the answer's token the likeliest one?
        score_case("score-512", "score", "bf16", 512, 2048, 50001, 1, ignored=0.375),
        # scoring a long document over a large ragged vocabulary, with alternatives
        score_case("score-4096", "score", "bf16", 4096, 2048, 100003, 20),
        # a small batch of sampled answers: the gradient of W is most of the traffic
        score_case("policy-64", "policy", "bf16", 64, 1024, 32000, 0),
        # an ordinary batch in f32, the type of the library's own solves
        score_case("policy-f32", "policy", "f32", 1024, 1024, 32000, 0),
        # a ragged batch of answers, the prompts' rows without a gradient
        score_case("policy-masked", "policy", "bf16", 2047, 1536, 50001, 0, ignored=0.375),
        # one small weight: latency
        orth_case("orth-128", "bf16", 1, 128, 128),
        # the attention heads' blocks of a model, each for itself
        orth_case("orth-heads", "f32", 200, 96, 64),
        # everything odd, in f32
        orth_case("orth-f32-odd", "f32", 1, 517, 1031),
        # the same weight of twelve layers, stacked
        orth_case("orth-layers", "bf16", 12, 1024, 4096),
        # the largest: a wide layer's weight, stored the other way round
        orth_case("orth-8192", "bf16", 1, 8192, 4096, turned=True),
    ]


def score_case(name, what, kind, rows, dim, vocab, top, ignored=0.0, pad=0):
    return {"name": name, "op": "score", "pass": what, "type": kind, "rows": rows, "dim": dim, "vocab": vocab, "top": top,
            "ignored": ignored, "pad": pad}


def orth_case(name, kind, batch, rows, cols, turned=False, steps=5):
    return {"name": name, "op": "orth", "type": kind, "batch": batch, "rows": rows, "cols": cols, "turned": turned, "steps": steps}


def log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.6:
        while True:
            rows, dim, vocab = log_between(rng, 1, 4096), log_between(rng, 64, 4096), log_between(rng, 2000, 131072)
            if rng.random() < 0.5:
                dim = -(-dim // 64) * 64
            if rows * dim * vocab * (6 if kind == "f32" else 1) <= 4096 * 2048 * 100003:
                break
        what = rng.choice(["score", "score", "policy"])
        c = score_case("", what, kind, rows, dim, vocab, rng.choice([0, 1, 5, 20]) if what == "score" else 0,
                       rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 2)]), rng.choice([0, 0, rng.randrange(1, 64)]))
    else:
        while True:
            batch, rows, cols = log_between(rng, 1, 256), log_between(rng, 16, 8192), log_between(rng, 16, 8192)
            if max(rows, cols) <= 8 * min(rows, cols) and batch * rows * cols * min(rows, cols) <= 4096 * 4096 * 4096:
                break
        if rng.random() < 0.5:
            rows, cols = -(-rows // 16) * 16, -(-cols // 16) * 16
        c = orth_case("", kind, batch, rows, cols, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return prepare_score(case, gen) if case["op"] == "score" else prepare_orth(case, gen)


def prepare_score(case, gen):
    """Hidden vectors and weights on the grid of fixed-point values (steps of 2^-6 and 2^-12), as they
    are after quantisation: logits are then whole multiples of 2^-18, and the order in which a sum is
    formed does not decide which of two close alternatives comes first."""
    rows, dim, vocab, kind = case["rows"], case["dim"], case["vocab"], TYPES[case["type"]]
    W = torch.randn(vocab, dim, device="cuda", generator=gen).mul_(4096 / math.sqrt(dim)).round_().div_(4096)
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    # rows of unit scale that lean towards their target's vector by a random amount, as a model's do
    lean = torch.rand(rows, 1, device="cuda", generator=gen) * 10
    H = torch.empty(rows, dim + case["pad"], device="cuda", dtype=kind)[:, :dim]
    H.copy_(((torch.randn(rows, dim, device="cuda", generator=gen) * 2 + lean * W[t]) * 64).round() / 64)
    skipped = torch.rand(rows, device="cuda", generator=gen) < case["ignored"]
    skipped[0] = False                                         # one row at least has a target
    t = torch.where(skipped, torch.full_like(t, -100), t)
    n = max(1, int((~skipped).sum()))
    # what a policy's loss gives: an advantage of either sign for each token, one small weight for the entropy
    g = torch.where(skipped, 0.0, torch.randn(rows, device="cuda", generator=gen) / n)
    e = torch.where(skipped, 0.0, -0.01 / n)
    return {"case": case, "H": H, "W": W.to(kind), "t": t, "g": g, "e": e}


def prepare_orth(case, gen):
    """Averaged gradients: a few strong directions, many weak ones, and noise."""
    batch, rows, cols = case["batch"], case["rows"], case["cols"]
    r = max(1, min(rows, cols) // 4)
    fall = torch.logspace(0, -3, r, device="cuda")
    G = (torch.randn(batch, rows, r, device="cuda", generator=gen) * fall) @ torch.randn(batch, r, cols, device="cuda", generator=gen)
    G += 0.1 * torch.randn(batch, rows, cols, device="cuda", generator=gen)
    G = (G * 1e-3).to(TYPES[case["type"]])
    if case["turned"]:
        G = G.transpose(1, 2).contiguous().transpose(1, 2)
    return {"case": case, "G": G if batch > 1 else G[0]}


# ------------------------------------------------------------------ one pass

def run(state):
    return run_score(state) if state["case"]["op"] == "score" else run_orth(state)


def run_score(state):
    H, W, t, g, e, case = state["H"], state["W"], state["t"], state["g"], state["e"], state["case"]
    if own:
        import matrix_dense_linear_spd_gb300 as bl
        logp, entropy, lse, top_logp, top_id = bl.score(H, W, t, case["top"])
        out = {"logp": logp, "entropy": entropy, "top_logp": top_logp, "top_id": top_id}
        if case["pass"] == "policy":
            out["dH"], out["dW"] = bl.score_grad(H, W, t, lse, entropy, g, e)
        return out
    counted = (t >= 0) & (t < W.shape[0])
    at = torch.where(counted, t, torch.zeros_like(t))[:, None]
    h, w = torch.where(counted[:, None], H.float(), 0.0), W.float()
    s = h @ w.T
    # the likeliest: the order of the values' bits as whole numbers, the lowest index first among equals
    bits = (s + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() * 2 ** 32 + (2 ** 32 - 1 - torch.arange(W.shape[0], device=s.device))
    top_id = 2 ** 32 - 1 - (key.topk(case["top"], 1).values & 0xffffffff)
    del key, bits
    top = s.amax(1, keepdim=True)
    x = s - (top + (s - top).exp().sum(1, keepdim=True).log())
    p = x.exp()
    entropy = -(p * x).sum(1)
    out = {"logp": torch.where(counted, x.gather(1, at)[:, 0], 0.0), "entropy": torch.where(counted, entropy, 0.0),
           "top_logp": torch.where(counted[:, None], x.gather(1, top_id), 0.0), "top_id": torch.where(counted[:, None], top_id, -1)}
    if case["pass"] == "policy":
        g, e = torch.where(counted, g, 0.0)[:, None], torch.where(counted, e, 0.0)[:, None]
        p = -p * (g + e * (x + entropy[:, None]))
        p.scatter_add_(1, at, g)
        out["dH"], out["dW"] = (p @ w).to(H.dtype), (p.T @ h).to(W.dtype)
    return out


COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def run_orth(state):
    G, steps = state["G"], state["case"]["steps"]
    if own:
        import matrix_dense_linear_spd_gb300 as bl
        return {"X": bl.orth(G, steps=steps, coefficients=COEFFICIENTS)}
    a, b, c = COEFFICIENTS
    X = G.float()
    turn = X.shape[-2] > X.shape[-1]
    if turn:
        X = X.transpose(-1, -2)
    X = X / X.square().sum((-2, -1), keepdim=True).sqrt()
    for _ in range(steps):
        A = X @ X.transpose(-1, -2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return {"X": (X.transpose(-1, -2) if turn else X).to(G.dtype)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    b = BYTES[case["type"]]
    if case["op"] == "orth":
        m, n = sorted((case["rows"], case["cols"]))
        # a step: X X^T and A A are symmetric, half of each is enough; then the product with X
        return {"bytes": 2 * case["batch"] * m * n * b, "flops": case["steps"] * case["batch"] * (3 * m * m * n + m * m * m)}
    rows, dim, vocab = case["rows"], case["dim"], case["vocab"]
    kept = max(1, round(rows * (1 - case["ignored"])))      # rows without a target are neither read nor multiplied
    if case["pass"] == "score":
        return {"bytes": (kept + vocab) * dim * b + rows * (16 + 12 * case["top"]), "flops": 2 * kept * dim * vocab}
    return {"bytes": (kept + rows + 2 * vocab) * dim * b + rows * 24, "flops": 6 * kept * dim * vocab}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return exact_score(s) if case["op"] == "score" else exact_orth(s)


def exact_score(s):
    case, t = s["case"], s["t"]
    rows, dim, vocab, k = case["rows"], case["dim"], case["vocab"], case["top"]
    if (2 if case["pass"] == "score" else 6) * rows * dim * vocab > 1.6e13:
        return None

    def zeros(*shape):
        return torch.zeros(*shape, device="cuda", dtype=torch.float64)
    W, logp, entropy, top_logp = s["W"].double(), zeros(rows), zeros(rows), zeros(rows, k)
    top_id = torch.full((rows, k), -1, device="cuda", dtype=torch.int64)
    dH, dW = zeros(rows, dim), torch.zeros_like(W)
    for r in ((t >= 0) & (t < vocab)).nonzero()[:, 0].split(512):
        h, each = s["H"][r].double(), torch.arange(len(r), device="cuda")
        ls = torch.log_softmax(h @ W.T, 1)
        p = ls.exp()
        logp[r] = ls[each, t[r]]
        entropy[r] = -(p * ls).sum(1)
        if k:
            value, place = torch.sort(h @ W.T, dim=1, descending=True, stable=True)
            top_id[r] = place[:, :k]
            top_logp[r] = ls.gather(1, place[:, :k])
        if case["pass"] == "policy":
            d = -s["g"][r, None].double() * p
            d[each, t[r]] += s["g"][r].double()
            d -= s["e"][r, None].double() * p * (ls + entropy[r, None])
            dH[r] = d @ W
            dW.addmm_(d.T, h)
    out = {"logp": logp, "entropy": entropy, "top_logp": top_logp, "top_id": top_id}
    return out if case["pass"] == "score" else {**out, "dH": dH, "dW": dW}


def exact_orth(s):
    case, G = s["case"], s["G"].double()
    m, n = sorted((case["rows"], case["cols"]))
    if case["batch"] * case["steps"] * (4.0 * m * m * n + 2.0 * m * m * m) > 1.2e13:
        return None
    a, b, c = COEFFICIENTS
    X = G / torch.linalg.vector_norm(G, dim=(-2, -1), keepdim=True)
    wide = case["rows"] <= case["cols"]
    for _ in range(case["steps"]):
        A = X @ X.mT if wide else X.mT @ X
        P = b * A + c * (A @ A)
        X = a * X + (P @ X if wide else X @ P)
    return {"X": X}
