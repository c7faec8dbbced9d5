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
@pytest.mark.parametrize("value", ["lowest"])
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
