"""MXFP4 on the GPU: what the calls do to the memory, streams and gradients around them."""
import pytest
import torch

from oracle import mx
from tests.test_gpu_mx import dense

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axes", ["rows", "columns", "both"])
@pytest.mark.parametrize("m,k", [(37, 75), (1, 33), (130, 1), (4129, 8225)])
def test_quantize_writes_zeros_behind_a_rows_last_scale(axes, m, k):
    """Up to the next multiple of 4 bytes, along either axis, and nothing behind it."""
    x = dense(m, k, torch.bfloat16, 200).cuda()

    def room(rows, depth):
        nb = mx.blocks(depth)
        held = torch.full((rows, (nb + 3) // 4 * 4 + 4), 0xA5, dtype=torch.uint8, device="cuda")
        return torch.empty(rows, 16 * nb, dtype=torch.uint8, device="cuda"), held, nb

    q, s, nk = room(m, k)
    qt, st, nm = room(k, m)
    rows, cols = (q, s[:, :nk]), (qt, st[:, :nm])
    fp4.fp4_quantize_mxfp4(m, k, x, *(rows if axes != "columns" else (None, None)), *(cols if axes != "rows" else (None, None)))
    for held, nb, on in ((s, nk, axes != "columns"), (st, nm, axes != "rows")):
        end = (nb + 3) // 4 * 4
        assert not held[:, nb:end].any() if on else (held == 0xA5).all()
        assert (held[:, end:] == 0xA5).all()
