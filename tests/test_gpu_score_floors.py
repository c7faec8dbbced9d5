"""Scores with alternatives: blocks of logits below their row's floor stay unwritten, whatever the tiles' width."""
import pytest

from _gpu import lib, torch_cuda
from test_gpu_xent import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,rows,vocab", [("f32", 128, 200000), ("f32", 9, 200000), ("bf16", 128, 200000), ("bf16", 300, 60000)])
@pytest.mark.parametrize("top", [1, 2, 5, 20, 32])
def test_blocks_below_the_floor_are_not_written(kind, rows, vocab, top):
    """Logits in random order. The tiles of the first round, a tenth of the vocabulary, know no floor. Of the others a
    block of 32 is kept if it reaches the least of `top` sets' maxima over what came before: at the end some top log(top)
    of 6250 (of 1875) blocks do, on the way 32 log(32) log(10) at most more. A quarter at least stays as it was."""
    torch, bl = torch_cuda(), lib()
    H, W, t, _ = make(rows, 64, vocab, kind, seed=top)
    raw, code = bl.get_lib(), bl.BL_F32 if kind == "f32" else bl.BL_BF16
    need = raw.bl_score_workspace(code, rows, 64, vocab, top, H.data_ptr(), 64, W.data_ptr(), 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    logp, entropy, lse = (torch.empty(rows, device="cuda") for _ in range(3))
    top_logp, top_id = torch.empty(rows, top, device="cuda"), torch.empty(rows, top, dtype=torch.int64, device="cuda")
    assert raw.bl_score(code, rows, 64, vocab, top, H.data_ptr(), 64, W.data_ptr(), 64, t.data_ptr(), logp.data_ptr(), entropy.data_ptr(),
                        lse.data_ptr(), top_logp.data_ptr(), top_id.data_ptr(), ws.data_ptr(), need,
                        torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    untouched = int((ws.view(torch.int32) == -1).sum())
    assert untouched >= rows * vocab // 4, untouched / (rows * vocab)
    # (values that come close in f32: the order of equal ones is the operator's own, tested elsewhere)
    want = (H.double() @ W.double().T).topk(top, 1).values - lse.double()[:, None]
    assert float((top_logp.double() - want).abs().amax()) < 1e-3
