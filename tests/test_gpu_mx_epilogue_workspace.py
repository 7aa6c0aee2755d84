"""MXFP4 products with an epilogue in workspaces of every size: K in as many parts as fit, right in all of them."""
import pytest
import torch

from tests import mx_reference as ref
from tests.mx_reference import dense, f64

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,act,residual", [(20, 635, 8192, None, False), (23, 1687, 8192, "silu", True), (80, 2176, 26080, None, False),
                                                (41, 688, 15840, "gelu", True)])
def test_as_many_parts_as_fit(m, n, k, act, residual):
    x, w = dense(m, k, torch.bfloat16, 1), fp4.MXTensor.quantize(dense(n, k, torch.float32, 2, scale=0.1))
    a, b = fp4.MXTensor.quantize(x), dense(1, n, torch.bfloat16, 3)[0]
    r = dense(m, n, torch.float32, 4) if residual else None
    kw = dict(bias=b, activation=act, residual=r)
    z, ez = ref.with_bias(*ref.product(ref.values(x), f64(w.dequant()), k), f64(b))
    want, tol = ref.out(z, ez, act, f64(r) if residual else None, torch.float32)
    e = fp4.Epilogue(b.data_ptr(), r.data_ptr() if residual else None, None, n, n, 2, 1, [None, "relu", "silu", "gelu"].index(act))
    need, any_ = fp4.lib().w4a4_matmul_epilogue_workspace_bytes(m, n, k, e), fp4.w4a4_matmul_workspace_bytes(m, n, k)
    assert any_ >= need > 0
    first, seen = w.matmul(a, **kw), []
    ref.check(first, want, tol)
    for size in (any_, need, need - 16, need // 2, need // 4 + 16, need // 8, 16):
        room = torch.empty(size // 16 * 16 + 64, dtype=torch.uint8, device="cuda").fill_(0xA5)
        y = w.matmul(a, workspace=room[:size // 16 * 16], **kw)
        assert (room[size // 16 * 16:] == 0xA5).all()
        ref.check(y, want, tol, f"{size}")
        if size >= need:
            assert torch.equal(y, first)
        seen.append(y)
    operand = fp4.lib().w4a4_linear_epilogue_workspace_bytes(m, n, k, e) - need
    for size in (0, need // 2 // 16 * 16, need):
        room = torch.empty(operand + size, dtype=torch.uint8, device="cuda").fill_(0xA5)
        y = w.matmul(x, workspace=room, **kw)
        ref.check(y, want, tol, f"linear {size}")
        if size == need:
            assert torch.equal(y, first)
    with pytest.raises(RuntimeError, match="w4a4_linear"):
        w.matmul(x, workspace=room[:operand - 256], **kw)
