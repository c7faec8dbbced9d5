"""Scores and their gradients, through the C ABI: a result that overlaps another tensor of the call is refused. All tensors
lie in one allocation, each in a slot that holds the largest of them; with these sizes no kernel takes an index from
memory unchecked, so a call that were let through would stay within it."""
import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu

ROWS, DIM, VOCAB, TOP = 8, 16, 64, 3
SCORE = ("H", "W", "target", "logp", "entropy", "lse", "top_logp", "top_id", "ws")
GRAD = ("H", "W", "target", "lse", "entropy", "g", "e", "dH", "dW", "ws")
PAIRS = [("score", a, b) for a in ("logp", "entropy", "lse", "top_logp", "top_id", "ws") for b in SCORE if SCORE.index(b) < SCORE.index(a)]
PAIRS += [("grad", a, b) for a in ("dH", "dW", "ws") for b in GRAD if GRAD.index(b) < GRAD.index(a)]


def call(what, kind, moved=None, by=0):
    torch, bl = torch_cuda(), lib()
    raw, code = bl.get_lib(), bl.BL_F32 if kind == "f32" else bl.BL_BF16
    need = max(raw.bl_score_workspace(code, ROWS, DIM, VOCAB, TOP, 1024, DIM, 2048, DIM),
               raw.bl_xent_workspace(code, ROWS, DIM, VOCAB, 1024, DIM, 2048, DIM, 1))
    names = SCORE if what == "score" else GRAD
    slot = 2 * ((need + 4095) // 4096 * 4096)
    held = torch.zeros(slot * (len(names) + 1), dtype=torch.uint8, device="cuda")
    base = (held.data_ptr() + 255) // 256 * 256
    at = {n: base + i * slot for i, n in enumerate(names)}
    if moved:
        at[moved[0]] = at[moved[1]] + by
    s = torch.cuda.current_stream().cuda_stream
    if what == "score":
        st = raw.bl_score(code, ROWS, DIM, VOCAB, TOP, at["H"], DIM, at["W"], DIM, at["target"], at["logp"], at["entropy"], at["lse"],
                          at["top_logp"], at["top_id"], at["ws"], need, s)
    else:
        st = raw.bl_score_grad(code, ROWS, DIM, VOCAB, at["H"], DIM, at["W"], DIM, at["target"], at["lse"], at["entropy"], at["g"], at["e"],
                               at["dH"], DIM, at["dW"], DIM, at["ws"], need, s)
    torch.cuda.synchronize()
    return st, raw.bl_last_error()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["score", "grad"])
def test_apart_they_run(what, kind):
    assert call(what, kind)[0] == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("what,a,b", PAIRS)
def test_a_shared_byte_is_refused(what, a, b, kind):
    st, why = call(what, kind, (a, b))
    assert st == 1 and b"overlaps" in why
    if a != "ws":                                  # the last whole element of b: rows of 8 f32 values and more
        st, why = call(what, kind, (a, b), by=ROWS * 4 - 8)
        assert st == 1 and b"overlaps" in why
