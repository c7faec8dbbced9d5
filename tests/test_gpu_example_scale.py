"""The training example: a weight's orthogonalised step has one scale, whichever of the two kinds of step takes it."""
import math

import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu


def close(a, b):
    """Moved by x and back by y: the weights' and the steps' roundings in f32."""
    return float((a.double() - b.double()).abs().amax()) <= 2.0 ** -20 * float(b.abs().amax() + 8)


def test_both_steps_scale_a_weight_alike():
    torch, bl = torch_cuda(), lib()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    (A, W), x, target = ex.problem(rows=300, vocab=200)
    counted = (target >= 0).float()
    h = torch.tanh(x @ A)
    _, lse = bl.xent(h, W, target)
    dh, dW = bl.xent_grad(h, W, target, lse, counted / counted.sum())
    moved = [A.clone(), W.clone()]
    ex.step(moved, x, target, lr=1.0, max_norm=math.inf, orth=True)
    assert close(A - moved[0], ex.orthogonal(x.T @ (dh * (1 - h * h))))
    assert close(W - moved[1], ex.orthogonal(dW))

    torch.manual_seed(5)
    action = torch.multinomial(torch.softmax(h @ W.T, 1), 1)[:, 0]
    reward = (action == target).float()
    advantage = reward - reward[target >= 0].mean()
    dA, dW, _ = ex.policy_gradients((A, W), x, torch.where(target >= 0, action, -1), advantage, 0.01)
    moved = [A.clone(), W.clone()]
    torch.manual_seed(5)
    ex.policy_step(moved, x, target, lr=1.0, max_norm=math.inf)
    assert close(moved[0] - A, ex.orthogonal(dA))
    assert close(moved[1] - W, ex.orthogonal(dW))
