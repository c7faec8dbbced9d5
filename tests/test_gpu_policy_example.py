"""The operators of a policy's training step run together, as the training example uses them: scores, their
gradients, orthogonalised and clipped steps."""
import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu


def plain(A, W, x, action, advantage, weight):
    """The objective in 64 bits, recorded by autograd."""
    torch = torch_cuda()
    counted = (action >= 0) & (action < W.shape[0])
    x = x.double()[counted]
    ls = torch.log_softmax(torch.tanh(x @ A) @ W.T, 1)
    logp = ls.gather(1, action[counted][:, None])[:, 0]
    entropy = -(ls.exp() * ls).sum(1)
    return (advantage.double()[counted] * logp + weight * entropy).mean()


@pytest.mark.parametrize("rows", [40, 700])
def test_gradients_of_the_objective(rows):
    """Against autograd in 64 bits: f32 products throughout, a relative 2-norm of 1e-5."""
    torch = torch_cuda()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    (A, W), x, target = ex.problem(rows=rows, vocab=333)
    W = W * 40                                                    # distributions that are not flat
    advantage = torch.randn(rows, device="cuda")
    dA, dW, _ = ex.policy_gradients((A, W), x, target, advantage, 0.05)
    a, w = A.double().requires_grad_(), W.double().requires_grad_()
    plain(a, w, x, target, advantage, 0.05).backward()
    assert float((dA - a.grad).norm() / a.grad.norm()) < 1e-5
    assert float((dW - w.grad).norm() / w.grad.norm()) < 1e-5


def test_gradient_against_differences():
    torch = torch_cuda()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    (A, W), x, target = ex.problem(rows=64, vocab=100)
    W = W * 40
    advantage = torch.randn(64, device="cuda")
    dA, dW, _ = ex.policy_gradients((A, W), x, target, advantage, 0.05)
    h = 1e-5
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        ea = torch.randn(A.shape, device="cuda", generator=gen).double()
        ew = torch.randn(W.shape, device="cuda", generator=gen).double()
        up, down = (float(plain(A.double() + s * h * ea, W.double() + s * h * ew, x, target, advantage, 0.05)) for s in (1, -1))
        formula = float((dA.double() * ea).sum() + (dW.double() * ew).sum())
        size = float((dA.double() * ea).abs().sum() + (dW.double() * ew).abs().sum())
        assert abs((up - down) / (2 * h) - formula) <= 1e-5 * size + 1e-7


def test_example_runs():
    torch = torch_cuda()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    params, x, target = ex.problem(rows=500, vocab=200)
    history = ex.train(steps=5, orth=True, given=(params, x, target))
    assert all(loss == loss and norm > 0 and info == 0 for loss, norm, info in history)
    logp, entropy, right = (float(v) for v in ex.evaluate(params, x, target))
    ls = torch.log_softmax(torch.tanh(x.double() @ params[0].double()) @ params[1].double().T, 1)[target >= 0]
    assert abs(logp - float(ls.gather(1, target[target >= 0][:, None]).mean())) < 1e-4
    assert abs(entropy + float((ls.exp() * ls).sum(1).mean())) < 1e-4 and 0 <= right <= 1
    before = [p.clone() for p in params]
    reward, entropy, norm = ex.policy_step(params, x, target, lr=0.1, max_norm=1.0)
    assert 0 <= float(reward) <= 1 and float(entropy) > 0
    moved = sum(float((p - b).double().square().sum()) for p, b in zip(params, before)) ** 0.5
    assert abs(moved - 0.1 * min(1.0, float(norm))) < 1e-4


def test_a_captured_step_is_the_step():
    """Score, gradients, orthogonalised and clipped update of a fixed batch in one graph, replayed on new values."""
    torch, bl = torch_cuda(), lib()
    gen = torch.Generator(device="cuda").manual_seed(0)
    H = torch.randn(300, 160, device="cuda", generator=gen)
    W = torch.randn(5000, 160, device="cuda", generator=gen) / 12
    t = torch.randint(0, 5000, (300,), device="cuda", generator=gen)
    g, e = torch.randn(300, device="cuda", generator=gen), torch.full((300,), 0.01, device="cuda")

    def step():
        logp, entropy, lse, top, ids = bl.score(H, W, t, 5)
        dH, dW = bl.score_grad(H, W, t, lse, entropy, g, e)
        x = bl.orth(dW)
        y = bl.orth(dW[:1200].view(10, 120, 160))
        norm = bl.gclip([x, y], 1.0)
        return logp, entropy, top, ids, dH, dW, x, y, norm
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    H.mul_(0.7)
    W.add_(0.01)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)
