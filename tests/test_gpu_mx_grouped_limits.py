"""The sizes at which the training path of experts is refused, and that it is refused and not wrong; and that inference goes on."""
import pytest
import torch

from tests import mx_reference as ref
from tests.mx_reference import dense

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu


def test_more_than_4_million_rows_of_weights():
    e, n, k, t = 512, 8200, 32, 40                                        # 8200 are padded to 8448: 4.3 million positions
    w = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
    w[3], w[511] = dense(n, k, torch.bfloat16, 1), dense(n, k, torch.bfloat16, 2)
    x = dense(t, k, torch.bfloat16, 3)
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[4:512], off[512] = 10, t
    y = fp4.mx_grouped_linear(x, w, off)
    for rows, expert in ((slice(0, 10), 3), (slice(10, t), 511)):
        z, ez = ref.product(ref.values(x[rows]), ref.values(w[expert]), k)
        ref.check(y[rows], *ref.out(z, ez, None, None, y.dtype))
    with pytest.raises(RuntimeError, match="fp4_quantize_mxfp4_grouped"):
        fp4.mx_grouped_linear(x.clone().requires_grad_(), w, off)
    # x needs none: the weights' gradients contract the rows alone
    g = dense(t, n, torch.bfloat16, 4)
    (dw,) = torch.autograd.grad(fp4.mx_grouped_linear(x, w.requires_grad_(), off), w, g)
    assert not dw[:3].any() and not dw[4:511].any()
    z, ez = ref.product(ref.values(g[10:].T), ref.values(x[10:].T), t - 10)
    ref.check(dw[511], z, ref.rounded(z, ez, dw.dtype))


def test_more_than_4_million_rows():
    e, n, k = 512, 8, 32
    t = (1 << 22) - 255 * e + 1                                           # one row too many: each expert may pad 255
    assert fp4.lib().fp4_grouped_depth(t + 255, e) > 1 << 22 >= fp4.lib().fp4_grouped_depth(t - 1, e)
    x, w = torch.ones(t + 255, k, dtype=torch.bfloat16, device="cuda"), torch.ones(e, n, k, dtype=torch.bfloat16, device="cuda")
    off = torch.linspace(0, t + 255, e + 1, device="cuda", dtype=torch.float64).long()
    assert (fp4.mx_grouped_linear(x, w, off) == k).all()
    with pytest.raises(RuntimeError, match="fp4_quantize_mxfp4_grouped"):
        fp4.mx_grouped_linear(x, w.clone().requires_grad_(), off)
    xs = x[:t - 1].clone().requires_grad_()
    off.clamp_(max=t - 1)
    wl = w.clone().requires_grad_()
    g = torch.ones(t - 1, n, dtype=torch.bfloat16, device="cuda")
    dx, dw = torch.autograd.grad(fp4.mx_grouped_linear(xs, wl, off), (xs, wl), g)
    assert (dx == n).all() and torch.equal(dw, (off[1:] - off[:-1])[:, None, None].expand_as(dw).to(dw.dtype))
