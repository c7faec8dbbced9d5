"""A block-preconditioned training step built from this library's operators: softmax cross entropy
and its gradients (xent, xent_grad), one SPD solve per 32-wide block of each weight's input
(posv), and clipping of the whole step to a global norm (gclip).

The model is a two-layer token classifier, h = tanh(x A), logits = h W^T over a vocabulary. The
gradient of a weight is preconditioned on its input side by the diagonal blocks of the input's
second moment, (X_b^T X_b / rows + mu I) S_b = G_b: one batch of 32 x 32 systems with as many
right-hand sides as the weight has outputs.

Usage:
  python -m matrix_dense_linear_spd_gb300.train_example [--steps 20] [--rows 4096] [--vocab 512]
"""
from __future__ import annotations

import argparse

import torch

import matrix_dense_linear_spd_gb300 as bl

BLOCK = 32


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


def step(params, x, target, lr, max_norm):
    """One training step in place. Returns (mean loss, norm of the preconditioned step, infos)."""
    A, W = params
    h = torch.tanh(x @ A)
    loss, lse = bl.xent(h, W, target)
    counted = (target >= 0) & (target < W.shape[0])
    g = counted.float() / counted.sum().clamp(min=1)
    dh, dW = bl.xent_grad(h, W, target, lse, g)
    dA = x.T @ (dh * (1 - h * h))
    step_A, info_A = precondition(x, dA)
    step_W, info_W = precondition(h, dW.T)
    norm = bl.gclip([step_A, step_W], max_norm)
    A.sub_(step_A, alpha=lr)
    W.sub_(step_W.T, alpha=lr)
    return (loss * g).sum(), norm, (info_A, info_W)


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


def train(steps=20, lr=10.0, max_norm=0.25, **sizes):
    params, x, target = problem(**sizes)
    history = []
    for _ in range(steps):
        loss, norm, infos = step(params, x, target, lr, max_norm)
        history.append((loss, norm, torch.stack([i.abs().sum() for i in infos]).sum()))
    return [(float(a), float(b), int(c)) for a, b, c in history]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=512)
    a = ap.parse_args(argv)
    for i, (loss, norm, info) in enumerate(train(a.steps, rows=a.rows, vocab=a.vocab)):
        print(f"step {i:3d}  loss {loss:.4f}  norm of the step before clipping {norm:8.3f}  failed pivots {info}")


if __name__ == "__main__":
    main()
