"""The training operators' cases: softmax cross entropy over a large vocabulary (loss, and loss
with gradients) and the global gradient norm with clipping.

`own = False` computes the plain form in elementary torch operations; `own = True` calls the
package. Sizes are generic: token counts from one to a few thousand, vocabularies of a few
thousand to 131,072 entries, gradient lists from a handful of small tensors to two gigabytes.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # scoring one token against a vocabulary of ordinary size: one pass over W, latency and bandwidth
        xent_case("loss-1", "loss", "bf16", 1, 1024, 32000),
        # everything odd, in f32: rows, dim and vocab are no multiples of anything, rows strided
        xent_case("loss-f32-odd", "loss", "f32", 77, 259, 5003, pad=5),
        # evaluating a long document over a large ragged vocabulary
        xent_case("loss-4096", "loss", "bf16", 4096, 2048, 100003),
        # a small training batch: the gradient of W is most of the traffic
        xent_case("step-64", "step", "bf16", 64, 1024, 32000),
        # an ordinary batch in f32, the type of the library's own solves
        xent_case("step-f32", "step", "f32", 1024, 1024, 32000),
        # a ragged fine-tuning batch: the prompts' rows (a good third) have no target
        xent_case("step-masked", "step", "bf16", 2047, 1536, 50001, ignored=0.375),
        # the largest: a long sequence, a wide model, a vocabulary of 2^17
        xent_case("step-4096", "step", "bf16", 4096, 4096, 131072),
        # the norm alone, of a small model's gradients (what a training loop logs)
        grads_case("norm-12", "norm", "f32", 12, 40_000, 3.0),
        # clipping few small tensors: latency
        grads_case("clip-24", "clip", "f32", 24, 300_000, 4.0),
        # a flat gradient buffer cut into many odd pieces: no piece starts on a vector boundary
        grads_case("clip-flat-400", "clip", "bf16", 400, 30_000_000, 4.0, flat=True),
        # layers' gradients in f32, norm below the limit: scaled by one
        grads_case("clip-f32-60", "clip", "f32", 60, 120_000_000, 0.5),
        # a large model's gradients in bf16, two gigabytes
        grads_case("clip-bf16-62", "clip", "bf16", 62, 1_000_000_000, 16.0),
    ]


def xent_case(name, what, kind, rows, dim, vocab, ignored=0.0, pad=0):
    return {"name": name, "op": "xent", "pass": what, "type": kind, "rows": rows, "dim": dim, "vocab": vocab,
            "ignored": ignored, "pad": pad}


def grads_case(name, what, kind, tensors, total, norm, flat=False):
    return {"name": name, "op": "grads", "pass": what, "type": kind, "tensors": tensors, "total": total, "norm": norm,
            "flat": flat}


def log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    if rng.random() < 0.6:
        what, kind = rng.choice(["loss", "step"]), rng.choice(["bf16", "bf16", "f32"])
        while True:
            rows, dim, vocab = log_between(rng, 1, 4096), log_between(rng, 64, 4096), log_between(rng, 2000, 131072)
            if rng.random() < 0.5:
                dim = -(-dim // 64) * 64
            if rows * dim * vocab * (6 if kind == "f32" else 1) <= 4096 * 4096 * 131072:
                break
        c = xent_case("", what, kind, rows, dim, vocab, rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 2)]),
                      rng.choice([0, 0, rng.randrange(1, 64)]))
    else:
        tensors = log_between(rng, 1, 60)
        flat = rng.random() < 0.3
        c = grads_case("", rng.choice(["norm", "clip", "clip"]), rng.choice(["f32", "bf16", "f16", "mixed"]),
                       tensors * 7 if flat else tensors, log_between(rng, 20_000, 500_000_000), rng.choice([0.5, 2.0, 30.0]), flat)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return prepare_xent(case, gen) if case["op"] == "xent" else prepare_grads(case, gen)


def prepare_xent(case, gen):
    rows, dim, vocab, kind = case["rows"], case["dim"], case["vocab"], TYPES[case["type"]]
    W = torch.randn(vocab, dim, device="cuda", generator=gen).mul_(1 / math.sqrt(dim))
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    # rows of unit scale that lean towards their target's vector by a random amount, as a model's do
    lean = torch.rand(rows, 1, device="cuda", generator=gen) * 10
    H = torch.empty(rows, dim + case["pad"], device="cuda", dtype=kind)[:, :dim]
    H.copy_(torch.randn(rows, dim, device="cuda", generator=gen) * 2 + lean * W[t])
    skipped = torch.rand(rows, device="cuda", generator=gen) < case["ignored"]
    skipped[0] = False                                         # one row at least has a target
    t = torch.where(skipped, torch.full_like(t, -100), t)
    g = (~skipped).float() / max(1, int((~skipped).sum()))     # the mean over the counted rows
    return {"case": case, "H": H, "W": W.to(kind), "t": t, "g": g}


def sizes(case):
    """Element counts of the tensors: over three decades, odd ones among them, that sum to the total."""
    rng = random.Random(case["tensors"] * 1000003 + case["total"])
    share = [math.exp(rng.uniform(0, 7)) for _ in range(case["tensors"])]
    n = [max(1, int(case["total"] * s / sum(share))) for s in share]
    return [k // 8 * 8 if i % 3 and k > 64 and not case["flat"] else k for i, k in enumerate(n)]


def prepare_grads(case, gen):
    counts = sizes(case)
    scale = case["norm"] / math.sqrt(sum(counts))
    kinds = [TYPES[("f32", "bf16")[i % 2] if case["type"] == "mixed" else case["type"]] for i in range(len(counts))]
    if case["flat"]:
        kinds = [kinds[0]] * len(counts)
        whole = torch.randn(sum(counts), device="cuda", generator=gen, dtype=torch.float32).mul_(scale).to(kinds[0])
        result = torch.empty_like(whole)
        return {"case": case, "x": list(whole.split(counts)), "y": list(result.split(counts)), "result": result}
    x = [torch.randn(k, device="cuda", generator=gen).mul_(scale).to(d) for k, d in zip(counts, kinds)]
    return {"case": case, "x": x, "y": [torch.empty_like(v) for v in x], "result": None}


# ------------------------------------------------------------------ one pass

def run(state):
    return run_xent(state) if state["case"]["op"] == "xent" else run_grads(state)


def run_xent(state):
    H, W, t, g, what = state["H"], state["W"], state["t"], state["g"], state["case"]["pass"]
    if own:
        import matrix_dense_linear_spd_gb300 as bl
        loss, lse = bl.xent(H, W, t)
        if what == "loss":
            return {"loss": loss, "lse": lse}
        dH, dW = bl.xent_grad(H, W, t, lse, g)
        return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}
    counted = (t >= 0) & (t < W.shape[0])
    at = torch.where(counted, t, torch.zeros_like(t))[:, None]
    h, w = torch.where(counted[:, None], H.float(), 0.0), W.float()
    s = h @ w.T
    top = s.amax(1, keepdim=True)
    lse = (top + (s - top).exp().sum(1, keepdim=True).log())[:, 0]
    loss = torch.where(counted, lse - s.gather(1, at)[:, 0], 0.0)
    if what == "step":
        p = (s - lse[:, None]).exp()
        p.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        p *= torch.where(counted, g, 0.0)[:, None]
        dH, dW = (p @ w).to(H.dtype), (p.T @ h).to(W.dtype)
        return {"loss": loss, "lse": torch.where(counted, lse, 0.0), "dH": dH, "dW": dW}
    return {"loss": loss, "lse": torch.where(counted, lse, 0.0)}


LIMIT = 1.0      # the norm that clipping keeps the gradients to


def run_grads(state):
    x, y, what = state["x"], state["y"], state["case"]["pass"]
    if own:
        import matrix_dense_linear_spd_gb300 as bl
        if what == "norm":
            return {"norm": bl.gnorm(x)}
        norm = bl.gclip(x, LIMIT, out=y)
    else:
        norm = torch.stack([v.float().square().sum() for v in x]).sum().sqrt()
        if what == "norm":
            return {"norm": norm}
        c = torch.where(norm.isfinite(), (LIMIT / norm).clamp(max=1.0), 1.0)
        y = [o.copy_(v.float() * c) for v, o in zip(x, y)]
    return {"norm": norm, "y": y if state["result"] is None else state["result"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "grads":
        n = sizes(case)
        size = [BYTES[("f32", "bf16")[i % 2] if case["type"] == "mixed" else case["type"]] for i in range(len(n))]
        if case["flat"]:
            size = [size[0]] * len(n)
        total, b = sum(n), sum(k * s for k, s in zip(n, size))
        return {"bytes": b + 4 if case["pass"] == "norm" else 2 * b + 4, "flops": (2 if case["pass"] == "norm" else 3) * total}
    rows, dim, vocab, b = case["rows"], case["dim"], case["vocab"], BYTES[case["type"]]
    kept = max(1, round(rows * (1 - case["ignored"])))      # rows without a target are neither read nor multiplied
    if case["pass"] == "loss":
        return {"bytes": (kept + vocab) * dim * b + rows * 16, "flops": 2 * kept * dim * vocab}
    return {"bytes": (kept + rows + 2 * vocab) * dim * b + rows * 20, "flops": 6 * kept * dim * vocab}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return exact_xent(s) if case["op"] == "xent" else exact_grads(s)


def exact_xent(s):
    case, t, g = s["case"], s["t"], s["g"].double()
    if (2 if case["pass"] == "loss" else 6) * case["rows"] * case["dim"] * case["vocab"] > 1.6e13:
        return None
    kept = ((t >= 0) & (t < case["vocab"])).nonzero()[:, 0]
    W, loss, lse = s["W"].double(), torch.zeros(len(t), device="cuda", dtype=torch.float64), torch.zeros(len(t), device="cuda", dtype=torch.float64)
    dH, dW = torch.zeros(len(t), case["dim"], device="cuda", dtype=torch.float64), torch.zeros_like(W)
    for r in kept.split(1024):
        h = s["H"][r].double()
        z = h @ W.T
        lse[r] = torch.logsumexp(z, 1)
        loss[r] = -torch.log_softmax(z, 1)[torch.arange(len(r), device="cuda"), t[r]]
        if case["pass"] == "step":
            z = torch.softmax(z, 1)
            z[torch.arange(len(r), device="cuda"), t[r]] -= 1
            z *= g[r, None]
            dH[r] = z @ W
            dW.addmm_(z.T, h)
    return {"loss": loss, "lse": lse} if case["pass"] == "loss" else {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


def exact_grads(s):
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(v.double())) ** 2 for v in s["x"]))
    if s["case"]["pass"] == "norm":
        return {"norm": norm}
    y = [v.double() * min(1.0, LIMIT / norm) for v in s["x"]]
    return {"norm": norm, "y": y if s["result"] is None else torch.cat(y)}
