"""The training example: the operators run together, the loss falls, every solve succeeds and the
step that is applied has a norm of at most the limit."""
import pytest

from _gpu import torch_cuda

pytestmark = pytest.mark.gpu


def test_example_trains():
    torch_cuda()
    from matrix_dense_linear_spd_gb300 import train_example
    history = train_example.train(steps=20, rows=1000, vocab=300)
    losses = [h[0] for h in history]
    assert all(info == 0 for _, _, info in history)
    assert all(norm == norm and norm > 0 for _, norm, _ in history)
    assert abs(losses[0] - 5.70) < 0.3                # about log(300) before training
    assert losses[-1] < 0.8 * losses[0] and losses[-1] < losses[10] < losses[0]


def test_applied_step_is_clipped_and_solves_its_systems():
    torch = torch_cuda()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    params, x, target = ex.problem(rows=512, vocab=100)
    before = [p.clone() for p in params]
    _, norm, infos = ex.step(params, x, target, lr=1.0, max_norm=0.25)
    assert float(norm) > 0.25
    moved = sum(float(((p - b).double() ** 2).sum()) for p, b in zip(params, before)) ** 0.5
    assert abs(moved / 0.25 - 1) < 1e-4               # f32 rounding of the parameters' update
    g = torch.randn(x.shape[1], 7, device="cuda")
    s, info = ex.precondition(x, g)
    assert int(info.abs().sum()) == 0
    xb = x.double().view(512, -1, 32).transpose(0, 1)
    m = xb.transpose(1, 2) @ xb / 512 + 1e-2 * torch.eye(32, device="cuda", dtype=torch.float64)
    back = (m @ s.double().view(-1, 32, 7)).reshape(-1, 7)
    # condition number below 1e3 (eigenvalues of a 512-sample moment): f32 residual
    assert float((back - g).norm() / g.norm()) < 1e-4
