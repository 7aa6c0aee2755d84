"""MXFP4 products in the large tiles against FP64 (on the GPU, from the operands' values): streams of tiles per workgroup, odd
and ragged stages, K in parts, the column split, every output type, strided outputs, NaN blocks, the layer."""
import pytest
import torch

from oracle import mx
from tests.mx_plan import LAYER_CASES, TILE_CASES
from tests.test_gpu_mx import EPS, TINY, dense

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu


def values(x):
    """What the MXFP4 form of x (blocks along its last axis) stands for, in FP64: on [0, 2), [2, 4) and [4, 8) scales
    the levels are 1/2, 1 and 2 scales apart, and the even multiple is the even code."""
    r, k = x.shape
    v = torch.zeros(r, (k + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.reshape(r, -1, 32)
    big = v.abs().amax(2, keepdim=True)
    power = torch.where(big > 0, (torch.frexp(big)[1] - 3).clamp_min(-127), -127).double().exp2()
    q = v.abs() / power
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0)).double()
    level = (torch.round(q / step) * step).clamp_max(6)
    return (torch.copysign(level, v) * power).reshape(r, -1)[:, :k]


def sums(a, b):
    """(A B^T, |A| |B|^T)"""
    return a @ b.T.contiguous(), a.abs() @ b.abs().T.contiguous()


def close(y, ref, mag, k):
    """As in the tests of small sizes: the FP32 sum's bound, then one rounding to the output's type."""
    tol = float(mx.sum_bound(k, 1.0)) * mag
    tol += EPS[y.dtype] * (ref.abs() + tol) + TINY[y.dtype]
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), f"{tuple(y.shape)} {y.dtype}: worst {float((err / tol).max())} of the tolerance"


def operands(m, n, k):
    """Rows of very different size, so that a tile's operands or scales in the place of another's show; products that
    stay inside FP16."""
    a, b = dense(m, k, torch.float32, 300).mul(0.02).cuda(), dense(n, k, torch.float32, 301).mul(0.02).cuda()
    return a, b, fp4.MXTensor.quantize(a), fp4.MXTensor.quantize(b)


@pytest.mark.parametrize("m,n,k", TILE_CASES)
def test_tiles(m, n, k):
    a, b, ta, tb = operands(m, n, k)
    ref, mag = sums(values(a), values(b))
    assert float(ref.abs().max()) < 60000
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
        tb.matmul(ta, out=y)
        close(y, ref, mag, k)
        assert torch.equal(y, tb.matmul(ta, out_dtype=dtype))      # the same bits every time
        del y
    if TILE_CASES[m, n, k][1] > 1:                                 # without a workspace K is one part
        y = torch.full((m, n), float("nan"), device="cuda")
        fp4.w4a4_matmul(m, n, k, ta.codes, ta.scales, tb.codes, tb.scales, y, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
        close(y, ref, mag, k)


STRIDED = [(8190, 8100, 1100), (8190, 8200, 1100), (4090, 4090, 1300), (1999, 2111, 1100), (299, 2001, 33000)]


@pytest.mark.parametrize("m,n,k", STRIDED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("left,right", [(3, 4), (8, 16)])
def test_tiles_into_part_of_a_larger_output(m, n, k, dtype, left, right):
    """Rows that begin off 16 bytes, and rows that begin on them with a stride: the same bits, and nothing around them."""
    _, _, ta, tb = operands(m, n, k)
    stride = (n + left + right + 7) // 8 * 8 + (left % 2)
    y = torch.full((m + 2, stride), 7.0, dtype=dtype, device="cuda")
    tb.matmul(ta, out=y[1:-1, left:left + n])
    assert torch.equal(y[1:-1, left:left + n], tb.matmul(ta, out_dtype=dtype))
    y[1:-1, left:left + n] = 7.0
    assert bool((y == 7).all())


@pytest.mark.parametrize("m,n,k", STRIDED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_tiles_with_nan_blocks(m, n, k, dtype):
    a, b, ta, tb = operands(m, n, k)
    clean = tb.matmul(ta, out_dtype=dtype)
    rows, cols = [0, 17, m // 2, m - 1], [1, 255, n // 2 + 3, n - 1]
    a[rows[0], k - 1], a[rows[1], 0], a[rows[2], k // 2], a[rows[3], k - 1] = float("nan"), float("inf"), float("-inf"), float("nan")
    for i, c in enumerate(cols):
        b[c, (i * k) // 4] = float("nan")
    y = fp4.MXTensor.quantize(b).matmul(fp4.MXTensor.quantize(a), out_dtype=dtype)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[rows] = True
    bad[:, cols] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("m,n,k", LAYER_CASES)
@pytest.mark.parametrize("types", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16)])
def test_layer_in_large_tiles(m, n, k, types):
    x = dense(m, k, types[0], 310).mul(0.02).cuda().requires_grad_()
    w = dense(n, k, types[1], 311).mul(0.02).cuda().requires_grad_()
    g = dense(m, n, types[0], 312).mul(0.02).cuda()
    y = fp4.mx_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), g)
    x, w = x.detach(), w.detach()
    close(y.detach(), *sums(values(x), values(w)), k)
    close(dx, *sums(values(g), values(w.T.contiguous())), n)
    close(dw, *sums(values(g.T.contiguous()), values(x.T.contiguous())), m)


@pytest.mark.parametrize("m,n,k", [(4090, 4090, 1300), (1999, 2111, 1100)])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_dense_activations_in_large_tiles(m, n, k, name):
    from tests.test_gpu_mx import TYPES
    x = dense(m, k, TYPES[name], 320).mul(0.02).cuda()
    b = fp4.MXTensor.quantize(dense(n, k, torch.float32, 321).mul(0.02).cuda())
    assert torch.equal(b.matmul(x), b.matmul(fp4.MXTensor.quantize(x)))
    close(b.matmul(x, out_dtype=torch.float16), *sums(values(x), b.dequant().double()), k)
