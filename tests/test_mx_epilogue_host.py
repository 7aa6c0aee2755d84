"""MXFP4 products with an epilogue and products of experts without a GPU: the oracle's pins, the refusals of the library and of
the binding (each fails on the host, before anything is launched), and which tiles the sizes of the GPU tests run with."""
import ctypes
import os
import shutil
import subprocess
import tempfile
import warnings

import numpy as np
import pytest
import torch

from oracle import mx
from tests.mx_epilogue_cases import GRADIENT_TILES, GROUPED_TILES

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")

OK, ARG, SHAPE, ALIGN, UNSUP = 0, -1, -2, -3, -4
FAKE = 1 << 20
F32, BF16, F16 = 1, 2, 3


# ------------------------------------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("name", mx.ACTIVATIONS)
def test_slopes_are_the_activations_differences(name):
    z = np.concatenate([np.linspace(-9, 9, 181), [-40.0, 40.0]]) + 1 / 64
    h = 2.0 ** -12
    up, down = mx.activation(name, z + h)[0], mx.activation(name, z - h)[0]
    # central differences are off by h^2 / 6 of a third derivative that stays below 2, and by rounding
    assert np.abs((up - down) / (2 * h) - mx.slope(name, z)[0]).max() < h * h / 3 + 1e-11


def test_activations_are_torchs():
    z = torch.linspace(-12, 12, 997, dtype=torch.float64)
    f = torch.nn.functional
    for name, want in (("relu", f.relu(z)), ("silu", f.silu(z)), ("gelu", f.gelu(z)), ("gelu_tanh", f.gelu(z, approximate="tanh"))):
        assert np.abs(mx.activation(name, z.numpy())[0] - want.numpy()).max() < 1e-14


def test_interval_holds_the_quantised_values():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 100)) * np.exp2(rng.integers(-3, 4, (40, 1)))
    x[0, 0], x[1, 5] = 2.0, 0.0
    for e in (0.0, 1e-3, 0.05):
        low, high = mx.quantize_interval(x - e, x + e)
        for shift in (-1, 0, 1):
            q = mx.dequant(*mx.quantize(x + shift * e), 100)
            assert (low <= q).all() and (q <= high).all()
    # a block whose every value may be anything in a wide range, many scales apart
    y = np.exp2(rng.uniform(-30, 0, (200, 32))) * rng.choice([-1.0, 1.0], (200, 32))
    low, high = mx.quantize_interval(np.minimum(y, 0), np.maximum(y, 0))
    for shift in range(0, 30, 3):
        q = mx.dequant(*mx.quantize(y * np.exp2(-shift * rng.random((200, 32)))), 32)
        assert (low <= q).all() and (q <= high).all()
    low, high = mx.quantize_interval(x, x)
    assert np.array_equal(low, high) and np.array_equal(low, mx.dequant(*mx.quantize(x), 100))


# ------------------------------------------------------------------------------------------------ the library

def _mx(q=FAKE, s=FAKE, ldq=16 * 4, lds=4):
    return fp4.Mx(q, s, ldq, lds)


def _epi(bias=None, residual=None, z=None, ldr=16, ldz=16, bias_type=BF16, residual_type=BF16, act=0):
    return fp4.Epilogue(bias, residual, z, ldr, ldz, bias_type, residual_type, act)


def _groups(offsets=FAKE, count=2, bits=32):
    return fp4.Groups(offsets, count, bits)


BAD_EPILOGUES = [(None, ARG), (_epi(act=-1), ARG), (_epi(act=5), ARG), (_epi(bias=FAKE, bias_type=0), ARG), (_epi(bias=FAKE, bias_type=9), ARG),
                 (_epi(residual=FAKE, residual_type=0), ARG), (_epi(residual=FAKE, ldr=15), SHAPE), (_epi(z=FAKE, ldz=15), SHAPE),
                 (_epi(bias=FAKE + 1), ALIGN), (_epi(bias=FAKE + 2, bias_type=F32), ALIGN), (_epi(residual=FAKE + 1), ALIGN),
                 (_epi(residual=FAKE + 2, residual_type=F32), ALIGN), (_epi(z=FAKE + 2), ALIGN), (_epi(residual=FAKE, ldr=(1 << 40) + 1), UNSUP),
                 (_epi(z=FAKE, ldz=(1 << 40) + 1), UNSUP)]


def test_structs_mirror_the_header():
    assert (ctypes.sizeof(fp4.Epilogue), ctypes.sizeof(fp4.Groups), ctypes.sizeof(fp4.Gradient)) == (56, 24, 32)


@pytest.mark.parametrize("linear", [False, True])
def test_epilogue_product_refusals(linear):
    def call(ty=BF16, M=3, N=16, K=128, a="ok", b="ok", e="ok", y=FAKE, ldy=16, ws=None, wsb=0, xty=BF16, x=FAKE, ldx=128):
        a, b = (_mx() if v == "ok" else v for v in (a, b))
        e = _epi(act=2) if isinstance(e, str) else e
        if linear:
            return fp4.lib().w4a4_linear_epilogue(xty, ty, M, N, K, x, ldx, b, e, y, ldy, ws, wsb, None)
        return fp4.lib().w4a4_matmul_epilogue(ty, M, N, K, a, b, e, y, ldy, ws, wsb, None)
    for e, status in BAD_EPILOGUES:
        assert call(e=e) == status
    assert call(ty=0) == ARG and call(y=None) == ARG and call(b=None) == ARG and call(b=_mx(q=None)) == ARG
    assert call(M=-1) == SHAPE and call(N=0) == SHAPE and call(K=0) == SHAPE and call(ldy=15) == SHAPE and call(b=_mx(ldq=48)) == SHAPE
    assert call(K=(1 << 22) + 1) == UNSUP and call(N=(1 << 30) + 1, e=_epi()) == UNSUP
    assert call(b=_mx(s=FAKE + 1)) == ALIGN and call(y=FAKE + 1) == ALIGN and call(ws=FAKE + 8, wsb=64) == ALIGN
    assert call(M=0, y=None, a=None, b=None, x=None) == OK
    if linear:
        assert call(xty=0) == ARG and call(x=None) == ARG and call(ldx=100) == SHAPE and call(x=FAKE + 1) == ALIGN
        assert call(M=100) == ARG and call(M=100, ws=FAKE, wsb=16) == ARG          # needs its workspace
    else:
        assert call(a=None) == ARG and call(a=_mx(ldq=32)) == SHAPE


@pytest.mark.parametrize("linear", [False, True])
def test_grouped_product_refusals(linear):
    def call(ty=BF16, T=3, N=16, K=128, g="ok", a="ok", b="ok", e=None, y=FAKE, ldy=16, ws=None, wsb=0, xty=BF16, x=FAKE, ldx=128):
        a, b = (_mx() if v == "ok" else v for v in (a, b))
        g = _groups() if isinstance(g, str) else g
        if linear:
            return fp4.lib().w4a4_grouped_linear(xty, ty, T, N, K, g, x, ldx, b, e, 0, y, ldy, ws, wsb, None)
        return fp4.lib().w4a4_grouped_matmul(ty, T, N, K, g, a, b, e, 0, y, ldy, None)
    for e, status in BAD_EPILOGUES[1:]:
        assert call(e=e) == status
    assert call(g=None) == ARG and call(g=_groups(offsets=None)) == ARG and call(g=_groups(bits=16)) == ARG
    assert call(g=_groups(count=0)) == SHAPE and call(g=_groups(count=513)) == UNSUP
    assert call(g=_groups(offsets=FAKE + 2)) == ALIGN and call(g=_groups(offsets=FAKE + 4, bits=64)) == ALIGN
    assert call(N=(1 << 22), g=_groups(count=512), ldy=1 << 22) == UNSUP                    # 2^31 weight rows
    assert call(ty=0) == ARG and call(y=None) == ARG and call(b=None) == ARG
    assert call(T=-1) == SHAPE and call(N=0) == SHAPE and call(K=0) == SHAPE and call(ldy=15) == SHAPE and call(b=_mx(ldq=48)) == SHAPE
    assert call(T=(1 << 30) + 1) == UNSUP and call(K=(1 << 22) + 1) == UNSUP
    assert call(b=_mx(q=FAKE + 8)) == ALIGN and call(y=FAKE + 1) == ALIGN
    assert call(T=0, y=None, a=None, b=None, x=None) == OK
    if linear:
        assert call(xty=0) == ARG and call(x=None) == ARG and call(ldx=100) == SHAPE and call(x=FAKE + 1) == ALIGN
        assert call(T=100) == ARG and call(T=100, ws=FAKE, wsb=16) == ARG
    query = fp4.lib().w4a4_grouped_linear_workspace_bytes
    assert query(-1, 16, 32, 2) == SHAPE and query(3, 16, 32, 0) == SHAPE and query(3, 16, 32, 513) == UNSUP and query(0, 16, 32, 2) == 0
    assert query(100, 16, 128, 2) >= 100 * (64 + 4)


def test_backward_pieces_refusals():
    def quantize(ty=BF16, T=6, K=128, x=FAKE, ldx=128, g="ok", rows="ok", cols=None, d=None, ws=None, wsb=0):
        g = _groups() if isinstance(g, str) else g
        rows = _mx() if isinstance(rows, str) else rows
        return fp4.lib().fp4_quantize_mxfp4_grouped(ty, T, K, x, ldx, g, rows, cols, d, ws, wsb, None)

    def grad(z=None, dbias=None, ldz=128, act=0, ty=F32):
        return fp4.Gradient(z, dbias, ldz, act, ty)
    assert quantize(ty=0) == ARG and quantize(g=None) == ARG and quantize(rows=None) == ARG and quantize(x=None) == ARG
    assert quantize(T=-1) == SHAPE and quantize(K=0) == SHAPE and quantize(ldx=127) == SHAPE and quantize(rows=_mx(ldq=48)) == SHAPE
    assert quantize(g=_groups(count=0)) == SHAPE and quantize(g=_groups(count=513)) == UNSUP and quantize(g=_groups(bits=8)) == ARG
    assert quantize(T=7, g=_groups(offsets=None)) == SHAPE                                  # 7 rows in 2 groups alike
    # 6 rows in 2 groups have 512 positions along the columns
    assert fp4.lib().fp4_grouped_depth(6, 2) == 512 and quantize(cols=_mx(ldq=240, lds=16)) == SHAPE and quantize(cols=_mx(ldq=256, lds=12)) == SHAPE
    assert quantize(T=1 << 23, cols=_mx(ldq=1 << 22, lds=1 << 22)) == UNSUP
    assert quantize(d=grad(act=5)) == ARG and quantize(d=grad(dbias=FAKE, ty=0)) == ARG and quantize(d=grad(dbias=FAKE)) == ARG
    assert quantize(d=grad(z=FAKE, ldz=127)) == SHAPE and quantize(d=grad(z=FAKE, ldz=(1 << 23) + 1)) == UNSUP
    assert quantize(d=grad(z=FAKE + 2)) == ALIGN and quantize(d=grad(dbias=FAKE + 2)) == ALIGN
    assert quantize(d=grad(dbias=FAKE), ws=FAKE + 8, wsb=1 << 20) == ALIGN and quantize(d=grad(dbias=FAKE), ws=FAKE, wsb=64) == ARG
    assert quantize(T=0, x=None) == OK
    depth, sums = fp4.lib().fp4_grouped_depth, fp4.lib().fp4_grouped_sums_bytes
    assert depth(-1, 2) == SHAPE and depth(3, 0) == SHAPE and depth(3, 513) == UNSUP and depth(0, 4) == 0
    assert [depth(t, e) for t, e in ((1, 1), (256, 1), (257, 1), (512, 2), (513, 3), (5, 100))] == [256, 256, 512, 768, 1024, 1280]
    assert sums(-1, 8, 2) == SHAPE and sums(3, 0, 2) == SHAPE and sums(300, 100, 1) == 2 * 2 * 100 * 4

    def gradient(ty=BF16, T=6, N=16, K=32, g="ok", a="ok", b="ok", dw=FAKE, ldw=32):
        a, b = (_mx(ldq=256, lds=16) if v == "ok" else v for v in (a, b))
        return fp4.lib().w4a4_grouped_gradient(ty, T, N, K, _groups() if isinstance(g, str) else g, a, b, dw, ldw, None)
    assert gradient(ty=0) == ARG and gradient(dw=None) == ARG and gradient(a=None) == ARG and gradient(g=None) == ARG
    assert gradient(ldw=31) == SHAPE and gradient(a=_mx(ldq=128, lds=16)) == SHAPE and gradient(N=0) == SHAPE
    assert gradient(T=1 << 23) == UNSUP and gradient(b=_mx(q=FAKE + 8, ldq=256, lds=16)) == ALIGN

    def product_t(ty=BF16, T=6, N=16, K=32, g="ok", a="ok", b="ok", y=FAKE, ldy=32):
        a = _mx() if a == "ok" else a
        b = _mx(ldq=256, lds=16) if b == "ok" else b
        return fp4.lib().w4a4_grouped_matmul_t(ty, T, N, K, _groups() if isinstance(g, str) else g, a, b, 0, y, ldy, None)
    assert product_t(ty=0) == ARG and product_t(y=None) == ARG and product_t(b=None) == ARG and product_t(g=None) == ARG
    assert product_t(ldy=31) == SHAPE and product_t(b=_mx(ldq=128, lds=16)) == SHAPE and product_t(T=-1) == SHAPE
    assert product_t(N=1 << 21, g=_groups(count=4)) == UNSUP and product_t(a=_mx(s=FAKE + 2)) == ALIGN
    assert product_t(T=0, y=None, a=None, b=None) == OK


# ------------------------------------------------------------------------------------------------ the binding

def _operand(rows, k):
    t = torch.zeros(rows, 16 * -(-k // 32) + 64, dtype=torch.uint8)
    return fp4.MXTensor(t[:, :16 * -(-k // 32)], t[:, -64:][:, :-(-k // 32)], rows, k)


def test_python_refusals():
    w, a, x = _operand(8, 64), _operand(3, 64), torch.zeros(3, 64)
    off = torch.tensor([0, 1, 3])
    for f in (lambda **kw: w.matmul(a, **kw), lambda **kw: w.matmul(x, **kw), lambda **kw: w.grouped_matmul(a, off, **kw),
              lambda **kw: w.grouped_matmul(x, off, **kw), lambda **kw: fp4.mx_linear(x, torch.zeros(8, 64), **kw)):
        for bad, error in ((dict(activation="swish"), ValueError), (dict(activation=""), ValueError)):
            with pytest.raises((error, ValueError)):
                f(**bad)
        with pytest.raises(ValueError, match="GPU"):
            f(activation="silu")
    with pytest.raises(ValueError, match="does not hold"):
        w.grouped_matmul(x, torch.tensor([0, 1, 2, 3]))                       # 8 rows for 3 experts
    for bad in (torch.tensor([0]), torch.tensor(3), torch.zeros(2, 2, dtype=torch.int32)):
        with pytest.raises(ValueError, match="offsets"):
            w.grouped_matmul(x, bad)
    with pytest.raises(ValueError, match="depths"):
        w.grouped_matmul(torch.zeros(3, 32), off)
    with pytest.raises(ValueError):
        fp4.mx_grouped_linear(x, torch.zeros(2, 4, 32), off)
    with pytest.raises(ValueError):
        fp4.mx_grouped_linear(x, torch.zeros(8, 64), off)
    with pytest.raises(TypeError):
        fp4.mx_grouped_linear(x.double(), torch.zeros(2, 4, 64), off)


def test_calls_without_a_gradient_refuse_tensors_that_require_one():
    w, a, x, y = _operand(8, 64), _operand(3, 64), torch.zeros(3, 64), torch.zeros(3, 8)
    off, leaf = torch.tensor([0, 3]), torch.zeros(3, 8, requires_grad=True)
    bias = torch.zeros(8, requires_grad=True)
    for call in (lambda: w.matmul(a, residual=leaf), lambda: w.matmul(x, residual=leaf), lambda: w.matmul(a, bias=bias),
                 lambda: w.grouped_matmul(a, off, residual=leaf), lambda: w.grouped_matmul(x, off, bias=bias[None]),
                 lambda: w.grouped_matmul(x.clone().requires_grad_(), off), lambda: w.grouped_matmul(a, off, out=leaf),
                 lambda: fp4.w4a4_matmul(3, 8, 64, a.codes, a.scales, w.codes, w.scales, y, bias=bias),
                 lambda: fp4.w4a4_linear(3, 8, 64, x, w.codes, w.scales, y, residual=leaf),
                 lambda: fp4.w4a4_grouped_matmul(3, 8, 64, a.codes, a.scales, w.codes, w.scales, off, leaf),
                 lambda: fp4.w4a4_grouped_linear(3, 8, 64, x, w.codes, w.scales, off, y, bias=bias[None])):
        with pytest.raises(RuntimeError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call()


def test_traces_are_refused():
    from torch.fx.experimental.proxy_tensor import make_fx
    w, x, off = _operand(4, 64), torch.zeros(4, 64), torch.tensor([0, 4])
    for call in (lambda x: w.matmul(x, activation="relu"), lambda x: w.grouped_matmul(x, off), lambda x: fp4.mx_linear(x, x, activation="gelu"),
                 lambda x: fp4.mx_grouped_linear(x, x[None], off)):
        with pytest.raises(RuntimeError, match="traced"), warnings.catch_warnings():
            warnings.simplefilter("ignore")
            torch.jit.trace(call, (x,), check_trace=False)
        with pytest.raises(RuntimeError, match="traced"):
            make_fx(call)(x)


# ------------------------------------------------------------------------------------------------ which tiles

SOURCE = """
#include "mx_plan.h"
extern "C" int grouped(int64_t T, int64_t N, int64_t K, int64_t E) { return mx::grouped_tile(T, N, K, E, 256); }
extern "C" int gradient(int64_t T, int64_t M, int64_t N, int64_t E) { return mx::gradient_tile(T, M, N, E, 256); }
extern "C" int with(int64_t M, int64_t N, int64_t K, int erf, int other, int residual, int z) {
  const mx::EpilogueCosts c = mx::epilogue_costs(erf, other, residual, z);
  return mx::plan_of(M, N, K, 256, true, c.of).tile;
}
"""


@pytest.fixture(scope="module")
def rules():
    folder = tempfile.mkdtemp(prefix="mx_rules")
    try:
        source, lib = os.path.join(folder, "rules.cpp"), os.path.join(folder, "rules.so")
        with open(source, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(os.path.dirname(fp4.__file__), "csrc"), source,
                        "-o", lib], check=True, capture_output=True)
        yield ctypes.CDLL(lib)
    finally:
        shutil.rmtree(folder)


def _call(f, *args):
    return f(*(ctypes.c_int64(a) for a in args))


def test_cases_run_the_tiles_they_are_meant_to(rules):
    for (t, n, k, e), tile in GROUPED_TILES.items():
        assert _call(rules.grouped, t, n, k, e) == tile, (t, n, k, e)
    for (t, m, n, e), tile in GRADIENT_TILES.items():
        assert _call(rules.gradient, t, m, n, e) == tile, (t, m, n, e)
    assert {*GROUPED_TILES.values()} == {0, 64, 96, 128, 256} and {*GRADIENT_TILES.values()} == {128, 256}


def test_a_heavy_epilogue_prefers_smaller_tiles(rules):
    size = [ctypes.c_int64(v) for v in (8192, 9728, 2560)]
    assert rules.__getitem__("with")(*size, 0, 0, 0, 0) == 256
    assert rules.__getitem__("with")(*size, 1, 0, 1, 0) == 128
