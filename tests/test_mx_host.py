"""MXFP4 without a GPU: the oracle's pins, and the library's refusals (every call here fails on the host, before
anything is launched)."""
import ctypes
import itertools
import warnings

import numpy as np
import pytest
import torch

from oracle import mx

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")

OK, ARG, SHAPE, ALIGN, UNSUP = 0, -1, -2, -3, -4
FAKE = 1 << 20
F32, BF16, F16 = 1, 2, 3


# ------------------------------------------------------------------------------------------------ the oracle

def test_levels_are_e2m1():
    # sign, two exponent bits (bias 1), one mantissa bit
    for code in range(8):
        e, m = code >> 1, code & 1
        assert mx.LEVELS[code] == ((1 + m / 2) * 2.0 ** (e - 1) if e else m / 2)


def test_quantize_hand_cases():
    x = np.zeros((1, 32))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26]
    codes, scales = mx.quantize(x)
    assert scales[0, 0] == 127                       # floor(log2 6) - 2 = 0
    got = mx.dequant(codes, scales)[0]
    assert got[:9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.5]   # halves go to the even code
    x[0, 9] = 7.9                                    # past 6 scales: saturates, and the scale stays
    codes, scales = mx.quantize(x)
    assert scales[0, 0] == 127 and mx.dequant(codes, scales)[0, 9] == 6.0
    x[0, 9] = 8.0
    assert mx.quantize(x)[1][0, 0] == 128
    assert mx.quantize(np.zeros((1, 5)))[1].tolist() == [[0]]
    assert mx.quantize(np.full((1, 5), 2.0 ** -140))[1].tolist() == [[0]]
    x[0, 3] = np.inf
    codes, scales = mx.quantize(x)
    assert scales[0, 0] == 255 and not codes.any() and np.isnan(mx.dequant(codes, scales)).all()


def test_quantize_is_nearest_by_brute_force():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 64)) * np.exp2(rng.integers(-20, 20, (4, 1)))
    codes, scales = mx.quantize(x)
    v = mx.dequant(codes, scales)
    for r, b in itertools.product(range(4), range(2)):
        blk, val = x[r, 32 * b:32 * b + 32], v[r, 32 * b:32 * b + 32]
        p = 2.0 ** (int(scales[r, b]) - 127)
        assert p <= np.abs(blk).max() / 4 < 2 * p
        grid = np.concatenate([mx.LEVELS, -mx.LEVELS]) * p
        assert np.array_equal(np.abs(blk - val), np.abs(blk[:, None] - grid).min(axis=1))


# ------------------------------------------------------------------------------------------------- refusals

def _mx(q=FAKE, s=FAKE, ldq=16 * 4, lds=4):
    return fp4.Mx(q, s, ldq, lds)


def _quantize(ty=BF16, M=3, K=128, x=FAKE, ldx=128, rows="ok", cols=None):
    rows = _mx() if rows == "ok" else rows
    return fp4.lib().fp4_quantize_mxfp4(ty, M, K, x, ldx, rows, cols, None)


def test_quantize_refusals():
    assert _quantize(ty=0) == ARG and _quantize(ty=4) == ARG
    assert _quantize(rows=None) == ARG
    assert _quantize(x=None) == ARG
    assert _quantize(rows=_mx(q=None)) == ARG and _quantize(rows=_mx(s=None)) == ARG
    assert _quantize(M=-1) == SHAPE and _quantize(K=0) == SHAPE
    assert _quantize(ldx=127) == SHAPE
    assert _quantize(rows=_mx(ldq=48)) == SHAPE and _quantize(K=160, ldx=160, rows=_mx(ldq=80, lds=4)) == SHAPE
    assert _quantize(K=(1 << 22) + 1, ldx=1 << 23) == UNSUP
    assert _quantize(rows=_mx(ldq=(1 << 22) + 16)) == UNSUP and _quantize(rows=_mx(lds=(1 << 22) + 4)) == UNSUP
    assert _quantize(x=FAKE + 1) == ALIGN and _quantize(ty=F32, x=FAKE + 2) == ALIGN
    assert _quantize(rows=_mx(q=FAKE + 8)) == ALIGN and _quantize(rows=_mx(ldq=72)) == ALIGN
    assert _quantize(rows=_mx(s=FAKE + 2)) == ALIGN and _quantize(rows=_mx(lds=6)) == ALIGN
    # along the columns the operand has K rows of depth M
    assert _quantize(M=64, cols=_mx(ldq=16)) == SHAPE
    assert _quantize(M=(1 << 22) + 1, cols=_mx(ldq=1 << 22, lds=1 << 22)) == UNSUP
    assert _quantize(M=0, x=None) == OK


def test_dequant_refusals():
    def call(ty=F32, M=3, K=128, a=None, out=FAKE, ldo=128):
        return fp4.lib().fp4_dequant_mxfp4(ty, M, K, a or _mx(), out, ldo, None)
    assert call(ty=F16) == ARG and call(out=None) == ARG and call(a=_mx(s=None)) == ARG
    assert call(ldo=100) == SHAPE and call(K=0) == SHAPE
    assert call(out=FAKE + 2) == ALIGN
    assert call(M=0, out=None) == OK


@pytest.mark.parametrize("linear", [False, True])
def test_product_refusals(linear):
    def call(ty=BF16, M=3, N=16, K=128, a="ok", b="ok", y=FAKE, ldy=16, ws=None, wsb=0, xty=BF16, x=FAKE, ldx=128):
        a, b = (_mx() if v == "ok" else v for v in (a, b))
        if linear:
            return fp4.lib().w4a4_linear(xty, ty, M, N, K, x, ldx, b, y, ldy, ws, wsb, None)
        return fp4.lib().w4a4_matmul(ty, M, N, K, a, b, y, ldy, ws, wsb, None)
    assert call(ty=0) == ARG and call(ty=7) == ARG
    assert call(y=None) == ARG and call(b=None) == ARG and call(b=_mx(q=None)) == ARG
    assert call(M=-1) == SHAPE and call(N=0) == SHAPE and call(K=0) == SHAPE and call(ldy=15) == SHAPE
    assert call(b=_mx(ldq=48)) == SHAPE and call(b=_mx(lds=0)) == SHAPE
    assert call(K=(1 << 22) + 1) == UNSUP and call(N=(1 << 30) + 1) == UNSUP and call(M=(1 << 30) + 1) == UNSUP
    assert call(b=_mx(s=FAKE + 1)) == ALIGN and call(y=FAKE + 1) == ALIGN and call(ws=FAKE + 8, wsb=64) == ALIGN
    assert call(M=0, y=None, a=None, b=None, x=None) == OK
    if linear:
        assert call(xty=0) == ARG and call(x=None) == ARG and call(ldx=100) == SHAPE and call(x=FAKE + 1) == ALIGN
        assert call(M=100, ldx=128) == ARG                       # needs its workspace
        need = fp4.lib().w4a4_linear_workspace_bytes(100, 16, 128)
        assert need > 0 and call(M=100, ws=FAKE, wsb=16) == ARG
    else:
        assert call(a=None) == ARG and call(a=_mx(q=FAKE + 4)) == ALIGN and call(a=_mx(ldq=32)) == SHAPE


def test_workspace_queries():
    q, ql = fp4.lib().w4a4_matmul_workspace_bytes, fp4.lib().w4a4_linear_workspace_bytes
    for f in (q, ql):
        assert f(-1, 16, 32) == SHAPE and f(1, 0, 32) == SHAPE and f(1, 16, 0) == SHAPE and f(1, 16, 1 << 23) == UNSUP
        assert f(0, 16, 32) == 0 and f(1, 4096, 4096) == 0
    assert q(8192, 14336, 4096) == 0                             # enough tiles: K is not split
    assert ql(300, 1000, 100) >= 300 * 64 + 300 * 4              # at least the quantised activations


def test_python_refusals():
    t = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fp4.MXTensor.empty(3, 0, device="cpu")
    with pytest.raises(TypeError):
        fp4.MXTensor.from_canonical(t.float(), t)
    with pytest.raises(ValueError):
        fp4.MXTensor.from_canonical(t, t[:3])
    with pytest.raises(ValueError):
        fp4.MXTensor.from_canonical(t, t)                        # 64 bytes are 128 values: 4 scales, not 64
    with pytest.raises(ValueError):
        fp4.MXTensor.from_canonical(t, t[:, :4])                 # not on a GPU
    with pytest.raises(TypeError):
        fp4.fp4_quantize_mxfp4(4, 64, torch.zeros(4, 64, dtype=torch.float64), t[:, :32], t[:, :2])
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        fp4.fp4_quantize_mxfp4(4, 64, x, t[:, :32], None)
    with pytest.raises(ValueError):
        fp4.fp4_quantize_mxfp4(4, 63, x, t[:, :32], t[:, :2])    # shape
    with pytest.raises(ValueError):
        fp4.fp4_quantize_mxfp4(64, 4, x.T, t[:, :32], t[:, :2])  # rows not contiguous
    with pytest.raises(ValueError):
        fp4.fp4_quantize_mxfp4(4, 64, x.as_strided((4, 64), (1, 1)), t[:, :32], t[:, :2])   # rows overlap
    with pytest.raises(ValueError):
        fp4.mx_linear(x, torch.zeros(8, 32))
    with pytest.raises(TypeError):
        fp4.mx_linear(x.double(), torch.zeros(8, 64))


def test_mx_struct_mirrors_the_header():
    assert ctypes.sizeof(fp4.Mx) == 32


def test_calls_without_a_gradient_refuse_tensors_that_require_one():
    t = torch.zeros(4, 64, dtype=torch.uint8)
    w = fp4.MXTensor(t[:, :32], t[:, :2], 4, 64)
    x, y = torch.zeros(3, 64), torch.zeros(3, 4)
    for leaf in (x.clone().requires_grad_(), x.clone().requires_grad_() * 2, x.T.clone().requires_grad_().T):
        with pytest.raises(RuntimeError, match="gradient"):
            w.matmul(leaf)
        with pytest.raises(RuntimeError, match="gradient"):
            fp4.w4a4_linear(3, 4, 64, leaf, w.codes, w.scales, y)
        for quiet in (leaf.detach(), x):
            with pytest.raises(ValueError, match="GPU"):                 # goes on to the next check
                w.matmul(quiet)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            w.matmul(leaf)
    out = y.clone().requires_grad_()
    for call in (lambda: w.matmul(w, out=out), lambda: w.matmul(x, out=out), lambda: fp4.w4a4_linear(3, 4, 64, x, w.codes, w.scales, out),
                 lambda: fp4.w4a4_matmul(3, 4, 64, w.codes, w.scales, w.codes, w.scales, out),
                 lambda: fp4.fp4_dequant_mxfp4(3, 4, w.codes, w.scales, out)):
        with pytest.raises(RuntimeError, match="gradient"):
            call()


def test_traces_are_refused():
    """A traced graph would hold the allocations without the kernels."""
    from torch.fx.experimental.proxy_tensor import make_fx
    t = torch.zeros(4, 64, dtype=torch.uint8)
    q, s = t[:, :32], t[:, :2]
    w = fp4.MXTensor(q, s, 4, 64)
    x, y = torch.zeros(4, 64), torch.zeros(4, 4)

    def into(call):
        def f(x):
            call(x)
            return x + 1
        return f

    calls = [lambda x: w.matmul(x), lambda x: w.matmul(w) + x[:, :4], lambda x: fp4.mx_linear(x, x),
             lambda x: fp4.MXTensor.quantize(x).codes, lambda x: fp4.MXTensor.quantize_both(x)[1].scales, lambda x: w.dequant() + x,
             into(lambda x: fp4.fp4_quantize_mxfp4(4, 64, x, q, s)),
             into(lambda x: fp4.fp4_dequant_mxfp4(4, 64, w.codes, w.scales, x)),
             into(lambda x: fp4.w4a4_linear(4, 4, 64, x, w.codes, w.scales, y)),
             into(lambda x: fp4.w4a4_matmul(4, 4, 64, w.codes, w.scales, w.codes, w.scales, y))]
    for call in calls:
        with pytest.raises(RuntimeError, match="traced"), warnings.catch_warnings():
            warnings.simplefilter("ignore")                              # torch.jit.trace is deprecated
            torch.jit.trace(call, (x,), check_trace=False)
        for mode in ("real", "fake"):
            with pytest.raises(RuntimeError, match="traced"):
                make_fx(call, tracing_mode=mode)(x)
    with pytest.raises(ValueError, match="GPU"):                         # outside a trace
        w.matmul(x)
