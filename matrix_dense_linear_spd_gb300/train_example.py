"""A block-preconditioned training step built from this library's operators: softmax cross entropy
and its gradients (xent, xent_grad), one SPD solve per 32-wide block of each weight's input
(posv), and clipping of the whole step to a global norm (gclip). With --orth the gradients are
orthogonalised (orth) in place of the solves. After training the model is scored (score) and improved
on its own samples by a few policy steps (score, score_grad, orth, gclip).

The model is a two-layer token classifier, h = tanh(x A), logits = h W^T over a vocabulary. The
gradient of a weight is preconditioned on its input side by the diagonal blocks of the input's
second moment, (X_b^T X_b / rows + mu I) S_b = G_b: one batch of 32 x 32 systems with as many
right-hand sides as the weight has outputs.

Usage:
  python -m matrix_dense_linear_spd_gb300.train_example [--steps 20] [--rows 4096] [--vocab 512] [--orth]
"""
from __future__ import annotations

import argparse

import torch

import matrix_dense_linear_spd_gb300 as bl

BLOCK = 32
SIDE = 1 << 16                # rows that one orthogonalisation takes


def precondition(x, grad, mu=1e-2):
    """S with (X_b^T X_b / rows + mu I) S_b = G_b for every block b of BLOCK inputs: x is
    (rows, inputs), grad (inputs, outputs). Returns S, and the solves' info."""
    rows, inputs = x.shape
    blocks = inputs // BLOCK
    xb = x.view(rows, blocks, BLOCK).transpose(0, 1)
    moment = (xb.transpose(1, 2) @ xb) / rows
    moment.diagonal(dim1=1, dim2=2).add_(mu)
    rhs = bl.colmajor(grad.reshape(blocks, BLOCK, -1))
    info = bl.posv(moment.transpose(1, 2), rhs)     # symmetric: the transposed view is column-major
    return rhs.reshape(inputs, -1), info


def orthogonal(grad):
    """The gradient with singular values of about 1, at the scale that a weight of its shape has: it is given as the
    weight is stored (turned it may have another scale). Rows beyond SIDE go in blocks, each by itself."""
    return torch.cat([bl.orth(b) * max(1.0, b.shape[0] / b.shape[1]) ** 0.5 for b in grad.split(SIDE)])


def step(params, x, target, lr, max_norm, orth=False):
    """One training step in place. Returns (mean loss, norm of the preconditioned step, infos)."""
    A, W = params
    h = torch.tanh(x @ A)
    loss, lse = bl.xent(h, W, target)
    counted = (target >= 0) & (target < W.shape[0])
    g = counted.float() / counted.sum().clamp(min=1)
    dh, dW = bl.xent_grad(h, W, target, lse, g)
    dA = x.T @ (dh * (1 - h * h))
    if orth:
        step_A, step_W = orthogonal(dA), orthogonal(dW).T
        info_A = info_W = torch.zeros(1, dtype=torch.int32, device=x.device)
    else:
        step_A, info_A = precondition(x, dA)
        step_W, info_W = precondition(h, dW.T)
    norm = bl.gclip([step_A, step_W], max_norm)
    A.sub_(step_A, alpha=lr)
    W.sub_(step_W.T, alpha=lr)
    return (loss * g).sum(), norm, (info_A, info_W)


def evaluate(params, x, target):
    """(mean log probability, mean entropy, share of rows whose target is the likeliest token) of the rows that count."""
    A, W = params
    logp, entropy, _, _, likeliest = bl.score(torch.tanh(x @ A), W, target, top=1)
    counted = (target >= 0) & (target < W.shape[0])
    n = counted.sum().clamp(min=1)
    return logp.sum() / n, entropy.sum() / n, (counted & (likeliest[:, 0] == target)).sum() / n


def policy_gradients(params, x, action, advantage, entropy_weight):
    """Gradients of the mean over the rows that count of advantage * logp(action) + entropy_weight * entropy:
    (dA, dW, mean entropy)."""
    A, W = params
    h = torch.tanh(x @ A)
    logp, entropy, lse, _, _ = bl.score(h, W, action)
    counted = (action >= 0) & (action < W.shape[0])
    share = counted.float() / counted.sum().clamp(min=1)
    dh, dW = bl.score_grad(h, W, action, lse, entropy, share * advantage, share * entropy_weight)
    return x.T @ (dh * (1 - h * h)), dW, (entropy * share).sum()


def policy_step(params, x, target, lr, max_norm, entropy_weight=0.01):
    """One step uphill in place: tokens sampled from the model, rewarded where they are the target."""
    A, W = params
    action = torch.multinomial(torch.softmax(torch.tanh(x @ A) @ W.T, 1), 1)[:, 0]
    reward = (action == target).float()
    action = torch.where(target >= 0, action, -1)
    dA, dW, entropy = policy_gradients(params, x, action, reward - reward[target >= 0].mean(), entropy_weight)
    step_A, step_W = orthogonal(dA), orthogonal(dW)
    norm = bl.gclip([step_A, step_W], max_norm)
    A.add_(step_A, alpha=lr)
    W.add_(step_W, alpha=lr)
    return reward[target >= 0].mean(), entropy, norm


def problem(rows=4096, inputs=128, hidden=64, vocab=512, seed=0):
    """Parameters to train, tokens, and the targets that a random teacher gives them (one in
    sixteen is left out)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * scale
    x = normal(rows, inputs)
    teacher = torch.tanh(x @ normal(inputs, hidden, scale=inputs ** -0.5)) @ normal(hidden, vocab)
    target = teacher.argmax(1)
    target[::16] = -1
    return [normal(inputs, hidden, scale=inputs ** -0.5), normal(vocab, hidden, scale=0.02)], x, target


def train(steps=20, lr=10.0, max_norm=0.25, orth=False, given=None, **sizes):
    params, x, target = given or problem(**sizes)
    history = []
    for _ in range(steps):
        loss, norm, infos = step(params, x, target, lr, max_norm, orth)
        history.append((loss, norm, torch.stack([i.abs().sum() for i in infos]).sum()))
    return [(float(a), float(b), int(c)) for a, b, c in history]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--orth", action="store_true", help="orthogonalise the gradients in place of the solves")
    a = ap.parse_args(argv)
    params, x, target = given = problem(rows=a.rows, vocab=a.vocab)
    for i, (loss, norm, info) in enumerate(train(a.steps, orth=a.orth, given=given)):
        print(f"step {i:3d}  loss {loss:.4f}  norm of the step before clipping {norm:8.3f}  failed pivots {info}")
    logp, entropy, right = evaluate(params, x, target)
    print(f"mean log probability {float(logp):.4f}  mean entropy {float(entropy):.4f}  likeliest token right {float(right):.3f}")
    for i in range(3):
        reward, entropy, norm = policy_step(params, x, target, lr=0.1, max_norm=1.0)
        print(f"policy step {i}  reward {float(reward):.3f}  entropy {float(entropy):.4f}  norm {float(norm):.3f}")


if __name__ == "__main__":
    main()
