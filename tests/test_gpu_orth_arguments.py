"""Orthogonalised steps through the C ABI: what the header says is not looked at."""
import ctypes

import pytest

from _gpu import lib, torch_cuda

pytestmark = pytest.mark.gpu

ABC = (3.4445, -4.7750, 2.0315)


def call(G, X, rows, cols, batch=1, ldg=None, ldx=None, ws=None, ws_bytes=0):
    torch, bl = torch_cuda(), lib()
    raw, code = bl.get_lib(), bl.BL_F32 if G.dtype == torch.float32 else bl.BL_BF16
    st = raw.bl_orth(code, rows, cols, batch, G.data_ptr(), rows if ldg is None else ldg, rows * cols, X.data_ptr(),
                     rows if ldx is None else ldx, rows * cols, 5, (ctypes.c_double * 3)(*ABC), ws, ws_bytes,
                     torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st


@pytest.mark.parametrize("rows,cols", [(40, 70), (128, 256), (256, 128)])
def test_a_workspace_that_is_not_needed_is_not_looked_at(rows, cols):
    """Neither where it points, into one of the matrices even, nor how large it is said to be."""
    torch, bl = torch_cuda(), lib()
    G = torch.randn(cols, rows, device="cuda")
    want = bl.orth(G)
    for ws, size in ((None, 0), (None, -1), (G.data_ptr() + 256, 0), (G.data_ptr() + 256, 1 << 40), (3, 7)):
        X = torch.zeros_like(G)
        assert call(G, X, rows, cols, ws=ws, ws_bytes=size) == 0, (ws, size, bl.get_lib().bl_last_error())
        assert torch.equal(X, want)


@pytest.mark.parametrize("rows", [50, 3000])
def test_one_column_has_no_leading_dimension(rows):
    torch, bl = torch_cuda(), lib()
    G = torch.randn(1, rows, device="cuda")
    want = bl.orth(G)
    need = bl.get_lib().bl_orth_workspace(bl.BL_F32, rows, 1, 1)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    for ld in (0, 1, -7, 1 << 40):
        X = torch.zeros_like(G)
        assert call(G, X, rows, 1, ldg=ld, ldx=ld, ws=ws.data_ptr(), ws_bytes=need) == 0, (ld, bl.get_lib().bl_last_error())
        assert torch.equal(X, want)
