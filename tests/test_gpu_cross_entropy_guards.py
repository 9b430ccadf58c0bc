"""The linear cross entropy given exactly its workspace and outputs, in every way through the products: what lies behind them stays
as it is, and the results are those of other buffers."""
import pytest
import torch

from moe_variable_size_amd import _lib, api
from tests.test_gpu_cross_entropy import BF, F32, make

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.mark.parametrize("M,K,V,dtype,off", [
    (1, 64, 5003, BF, 0), (12, 128, 3001, BF, 0),                        # few rows: logits in memory, dl in two parts
    (130, 64, 333, BF, 0), (300, 264, 20011, BF, 0),                     # tiles, dl in two parts
    (600, 264, 5003, BF, 0), (2049, 128, 8191, BF, 0),                   # tiles, dl without the rows' factor
    (300, 65, 3001, BF, 0), (700, 65, 3001, BF, 0), (640, 64, 1003, BF, 1),  # staged: odd rows, off 16-byte lines
    (64, 8192, 500, BF, 0), (600, 4096, 260, BF, 0),                     # reductions in ranges
    (4096, 64, 40001, BF, 0), (300, 32, (1 << 19) + 9, BF, 0),           # pieces, the last one short
    (70, 33, 300, F32, 0), (777, 101, 5003, F32, 0),                     # fp32 by parts, whole
    (33, 4100, 700, F32, 0), (200, 2633, 900, F32, 1),                   # in ranges, the logits in memory
    (12, 40, 5003, F32, 0), (40, 3, 501, F32, 0), (40, 64, 3, F32, 0),   # few rows, short rows, few columns
    (3000, 24, 50003, F32, 0),                                           # pieces
])
def test_nothing_behind_the_buffers_changes(M, K, V, dtype, off):
    x, W, t, g = make(M, K, V, dtype, seed=M + V)
    if off:
        x = torch.empty(M * K + off, dtype=dtype, device="cuda")[off:].view(M, K).copy_(x)
    lib, code, st = _lib.load(), 1 if dtype == BF else 0, torch.cuda.current_stream().cuda_stream

    def space(n):
        return torch.full((n + GUARD,), 0xAB, dtype=torch.uint8, device="cuda"), n

    outs = [torch.full((n + 512,), 7.0, dtype=d, device="cuda") for n, d in ((M, F32), (M, F32), (3, F32), (M * K, dtype), (V * K, dtype))]
    loss, lse, total, dX, dW = outs
    ws, n = space(lib.moe_linear_ce_fwd_workspace_bytes(M, K, V, code))
    assert lib.moe_linear_ce_fwd(x.data_ptr(), W.data_ptr(), t.data_ptr(), 64, M, K, V, 1e-3, loss.data_ptr(), lse.data_ptr(),
                                 total.data_ptr(), code, ws.data_ptr(), n, st) == 0
    assert (ws[n:] == 0xAB).all()
    sums = torch.empty(3, device="cuda")
    want = api.moe_linear_ce_fwd(x, W, t, z_weight=1e-3, total=sums)
    for reduction, name in enumerate(("none", "sum", "mean")):
        up = g if reduction == 0 else g[:1]
        ws, n = space(lib.moe_linear_ce_bwd_workspace_bytes(M, K, V, code))
        assert lib.moe_linear_ce_bwd(up.data_ptr(), reduction, total.data_ptr(), x.data_ptr(), W.data_ptr(), t.data_ptr(), 64,
                                     lse.data_ptr(), M, K, V, 1e-3, dX.data_ptr(), dW.data_ptr(), code, ws.data_ptr(), n, st) == 0
        assert (ws[n:] == 0xAB).all()
        back = api.moe_linear_ce_bwd(up, x, W, t, want[1], z_weight=1e-3, reduction=name, total=sums)
        for a, b in zip(outs, want + (sums,) + back):
            assert torch.equal(a[:b.numel()], b.flatten()) and (a[b.numel():] == 7).all(), name
