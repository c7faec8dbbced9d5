"""Cross entropy over a vocabulary part of which is masked: entries of W whose logits are the type's
lowest value or minus infinity in rows that count. A masked entry's probability is exactly 0, so the
loss and the gradients are those of the vocabulary without it, within the bounds of test_gpu_xent,
and dW is exactly zero for the entry itself.

The mask is one column: H holds +1 (or -1) there and W 0, or the mask's value for a masked entry. With
minus infinity dH is 0 * inf = NaN in that column, by the formula, and only there."""
import math

import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import check, make, reference

pytestmark = pytest.mark.gpu

VOCAB = 700


def masks(torch):
    v = torch.arange(VOCAB, device="cuda")
    return {"first": v < 160, "one": v == 3, "middle": (v >= 256) & (v < 520), "last": v >= 500, "most": v != 411,
            "odd": v % 2 == 1}


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 8, 100, 300])
@pytest.mark.parametrize("value", ["lowest", "-inf"])
@pytest.mark.parametrize("sign", [1, -1])
def test_masked_entries_have_no_share(kind, rows, value, sign):
    torch, bl = torch_cuda(), lib()
    for n, (name, masked) in enumerate(masks(torch).items()):
        H, W, t, g = make(rows, 73, VOCAB, kind, seed=rows + n)
        kept = (~masked).nonzero()[:, 0]
        t = kept[t % len(kept)]
        H[:, -1] = sign
        W[:, -1] = 0
        W[masked, -1] = sign * (torch.finfo(W.dtype).min if value == "lowest" else -math.inf)
        loss, lse = bl.xent(H, W, t)
        place = torch.zeros(VOCAB, dtype=torch.int64, device="cuda")
        place[kept] = torch.arange(len(kept), device="cuda")
        ref = reference(H, W[kept], place[t], g, kind)
        check(lse, ref, "lse")
        check(loss, ref, "loss")
        dH, dW = bl.xent_grad(H, W, t, lse, g)
        assert bool((dW[masked] == 0).all()), name
        check(dW[kept], ref, "dW")
        check(dH[:, :-1], {"dH": [x[:, :-1] for x in ref["dH"]]}, "dH")
        if value == "lowest":
            assert bool((dH[:, -1] == 0).all()), name


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 100, 300])
def test_a_mask_that_leaves_nothing(kind, rows):
    """Every entry at the lowest value: they share the row evenly, so the loss is log(vocab), within f32's rounding
    of the sum and the logarithm; lse is the lowest value to f32's precision. With minus infinity there
    is no softmax: NaN. Either way other rows are as they are without it."""
    torch, bl = torch_cuda(), lib()
    H, W, t, g = make(rows, 64, VOCAB, kind, seed=1)
    H[:, -1] = 0
    H[0] = 0
    H[0, -1] = 1
    low = torch.finfo(W.dtype).min
    W[:, -1] = low
    loss, lse = bl.xent(H, W, t)
    assert abs(float(loss[0]) / math.log(VOCAB) - 1) < 2.0 ** -18
    assert abs(float(lse[0]) / low - 1) < 2.0 ** -22
    if rows > 1:
        rest = reference(H[1:], torch.cat([W[:, :-1], torch.zeros_like(W[:, :1])], 1), t[1:], g[1:], kind)
        check(loss[1:], rest, "loss")
        check(lse[1:], rest, "lse")
    W[:, -1] = -math.inf
    H[1:, -1] = 1
    assert bool(bl.xent(H, W, t)[0].isnan().all())
