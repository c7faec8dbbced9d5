"""The training example with a vocabulary beyond what one orthogonalisation takes (sides of up to 2^16)."""
import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu


def test_long_weights_go_in_blocks():
    torch, bl = torch_cuda(), lib()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    grad = torch.randn(65536 + 300, 64, device="cuda")
    got = ex.orthogonal(grad)
    assert got.shape == grad.shape
    assert torch.equal(got[:65536], bl.orth(grad[:65536]) * 32.0)
    assert torch.equal(got[65536:], bl.orth(grad[65536:]) * (300 / 64) ** 0.5)
    assert torch.equal(ex.orthogonal(grad[:500]), bl.orth(grad[:500]) * (500 / 64) ** 0.5)
    assert torch.equal(ex.orthogonal(grad[:40]), bl.orth(grad[:40]))


@pytest.mark.parametrize("orth", [False, True])
def test_the_example_runs(orth, capsys):
    torch_cuda()
    from matrix_dense_linear_spd_gb300 import train_example as ex
    ex.main(["--vocab", "70000", "--rows", "200", "--steps", "2"] + (["--orth"] if orth else []))
    out = capsys.readouterr().out
    assert out.count("loss") == 2 and out.count("policy step") == 3 and "nan" not in out
