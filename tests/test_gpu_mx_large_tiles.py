"""MXFP4 products in tiles of 256 with an epilogue, dense and of experts, against FP64: every way out of a tile, outputs that the caches
hold and larger ones, and weight gradients whose groups have from none to five stages. A sample of rows, on the tiles' edges and
between them, is compared, with all its columns."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mx
from tests import mx_large_tile_cases as cases
from tests import mx_reference as ref
from tests.mx_reference import TYPES, dense, f64

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
NATIVE = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}


def operand(rows, k, *key, low=122):
    """Any codes, and scales of a few powers of two."""
    gen = torch.Generator("cuda").manual_seed(hash((rows, k, *key)) % (1 << 31))
    codes = torch.randint(0, 256, (rows, 16 * -(-k // 32)), dtype=torch.uint8, device="cuda", generator=gen)
    if k % 32:
        codes[:, k // 2 + k % 2:] = 0
        if k % 2:
            codes[:, k // 2] &= 15
    scales = torch.randint(low, low + 4, (rows, -(-k // 32)), dtype=torch.uint8, device="cuda", generator=gen)
    return fp4.MXTensor.from_canonical(codes, scales, k)


def some_rows(m, *key, every=256):
    r = np.random.default_rng([m, *key])
    edges = [i for t in range(0, m, every) for i in (t, t + 15, t + 16, t + 127, t + 128, t + 255) if i < m]
    picked = set(r.choice(edges, min(len(edges), 40), replace=False)) | set(r.integers(0, m, 40)) | {0, 1, m - 2, m - 1}
    return np.array(sorted(picked))


def sums(va, vb, k):
    """FP64 sums and how far FP32 ones may be off, of rows of A (values on the GPU)."""
    return torch.mm(va, vb.T).cpu().numpy(), mx.sum_bound(k, torch.mm(va.abs(), vb.abs().T).cpu().numpy())


def native(t):
    return fp4.Mx(t.codes.data_ptr(), t.scales.data_ptr(), t.codes.stride(0), t.scales.stride(0))


def wide_output(m, n, dtype):
    """(an m x n output inside a wider tensor, the tensor), rows aligned to 4 bytes."""
    held = torch.full((m, n + 6), 7.0, dtype=dtype, device="cuda")
    return held[:, 2:2 + n], held


@pytest.mark.parametrize("m,n,k", cases.DENSE)
def test_dense(m, n, k):
    a, b = operand(m, k, 1), operand(n, k, 2, low=120)
    rows = some_rows(m, 3)
    at = torch.from_numpy(rows).cuda()
    bare, bound = sums(a.dequant()[at].double(), b.dequant().double(), k)
    for i, (name, bias_type, residual_type, keep, out) in enumerate(cases.EPILOGUES):
        bias = None if bias_type is None else dense(1, n, TYPES[bias_type], 4, i)[0]
        residual = None if residual_type is None else torch.randn(m, n, device="cuda").to(TYPES[residual_type])
        y, held = wide_output(m, n, TYPES[out])
        z, held_z = wide_output(m, n, torch.float32) if keep else (None, None)
        e = fp4.Epilogue(None if bias is None else bias.data_ptr(), None if residual is None else residual.data_ptr(),
                         z.data_ptr() if keep else None, n, n + 6, NATIVE.get(None if bias is None else bias.dtype, 0),
                         NATIVE.get(None if residual is None else residual.dtype, 0), ACTS.index(name))
        rc = fp4.lib().w4a4_matmul_epilogue(NATIVE[y.dtype], m, n, k, native(a), native(b), e, y.data_ptr(), n + 6, None, 0,
                                            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        label = f"{m} {n} {k} {cases.EPILOGUES[i]}"
        s, es = ref.with_bias(bare, bound, None if bias is None else f64(bias))
        ref.check(y[at], *ref.out(s, es, name, None if residual is None else f64(residual[at]), y.dtype), label=label)
        if keep:
            ref.check(z[at], s, es, label + " z")
        for t in (held, held_z) if keep else (held,):
            assert (t[:, :2] == 7).all() and (t[:, -4:] == 7).all(), label
        # the same through the public call, which has rows of its own
        if not keep:
            again = b.matmul(a, out_dtype=y.dtype, bias=bias, activation=name, residual=residual)
            assert torch.equal(again, y), label


@pytest.mark.parametrize("sizes,n,k,outside", cases.GROUPED)
def test_experts(sizes, n, k, outside):
    front, behind = outside
    e, t = len(sizes), sum(sizes) + front + behind
    off = np.concatenate([[0], np.cumsum(sizes)]) + front
    offsets = torch.from_numpy(off).int().cuda()
    a, w = operand(t, k, 5), operand(e * n, k, 6, low=120)
    rows = some_rows(t, 7)
    rows = np.unique(np.concatenate([rows, off[:-1].clip(max=t - 1), (off[1:] - 1).clip(min=0)]))
    expert = np.searchsorted(off, rows, side="right") - 1
    inside = (rows >= off[0]) & (rows < off[-1])
    at = torch.from_numpy(rows).cuda()
    bare, bound = np.zeros((len(rows), n)), np.zeros((len(rows), n))
    for i in range(e):
        of = inside & (expert == i)
        if of.any():
            vb = fp4.MXTensor(w.codes[i * n:(i + 1) * n], w.scales[i * n:(i + 1) * n], n, k).dequant().double()
            bare[of], bound[of] = sums(a.dequant()[at[torch.from_numpy(of)]].double(), vb, k)
    for i, (name, bias_type, residual_type, out) in enumerate(cases.GROUPED_EPILOGUES):
        bias = None if bias_type is None else dense(e, n, TYPES[bias_type], 8, i)
        residual = None if residual_type is None else torch.randn(t, n, device="cuda").to(TYPES[residual_type])
        y = w.grouped_matmul(a, offsets, out_dtype=TYPES[out], bias=bias, activation=name, residual=residual)
        label = f"{sizes} {n} {k} {cases.GROUPED_EPILOGUES[i]}"
        s, es = ref.with_bias(bare, bound, None if bias is None else f64(bias)[expert.clip(0, e - 1)])
        r = None if residual is None else f64(residual[at])
        want, tol = ref.out(s, es, name, r, y.dtype)
        want[~inside] = 0 if r is None else r[~inside]
        tol[~inside] = ref.rounded(want[~inside], 0 * want[~inside], y.dtype)
        ref.check(y[at], want, tol, label)
        # into a wider tensor: the same, rows of no expert and what lies beside left alone
        wide, held = wide_output(t, n, y.dtype)
        w.grouped_matmul(a, offsets, out=wide, bias=bias, activation=name, residual=residual)
        assert torch.equal(wide[front:t - behind], y[front:t - behind]), label
        assert (held[:, :2] == 7).all() and (held[:, -4:] == 7).all() and (held[:front] == 7).all() and (held[t - behind:] == 7).all()


@pytest.mark.parametrize("sizes,outside,m,n", cases.GRADIENTS)
def test_weight_gradients(sizes, outside, m, n):
    front, behind = outside
    e, t = len(sizes), sum(sizes) + front + behind
    off = np.concatenate([[0], np.cumsum(sizes)]) + front
    offsets = torch.from_numpy(off).int().cuda()
    x, g = dense(t, n, torch.bfloat16, 9), dense(t, m, torch.bfloat16, 10)
    rows = some_rows(m, 11)
    at = torch.from_numpy(rows).cuda()
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        w = torch.zeros(e, m, n, dtype=dtype, device="cuda", requires_grad=True)
        y = fp4.mx_grouped_linear(x, w, offsets)
        (dw,) = torch.autograd.grad(y, w, g, retain_graph=True)
        assert dw.dtype == dtype and dw.shape == w.shape
        for i, (lo, hi) in enumerate(zip(off, off[1:])):
            if lo == hi:
                assert not dw[i].any()
                continue
            va, vb = ref.values(g[lo:hi, at].T), ref.values(x[lo:hi].T)
            want, tol = ref.product(va, vb, hi - lo)
            ref.check(dw[i][at], want, ref.rounded(want, tol, dtype), f"{sizes} {m} {n} {dtype} {i}")
        for _ in range(2):
            assert torch.equal(torch.autograd.grad(y, w, g, retain_graph=True)[0], dw)
        del w, y, dw


def test_layer_of_experts_keeps_its_sums():
    """A training step whose forward product keeps z in tiles of 256, against the same step expert by expert."""
    sizes, n, k = (4000, 0, 257, 3043), 4094, 4352
    e, t = len(sizes), sum(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)])
    x, g = dense(t, k, torch.bfloat16, 12), dense(t, n, torch.bfloat16, 13)
    w = (dense(e * n, k, torch.bfloat16, 14, scale=0.02)).reshape(e, n, k).requires_grad_()
    b = dense(e, n, torch.float32, 15).requires_grad_()
    y = fp4.mx_grouped_linear(x, w, torch.from_numpy(off).cuda(), bias=b, activation="gelu_tanh")
    dw, db = torch.autograd.grad(y, (w, b), g)
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo == hi:
            assert not dw[i].any() and not db[i].any()
            continue
        wi, bi = w[i].detach().requires_grad_(), b[i].detach().requires_grad_()
        yi = fp4.mx_linear(x[lo:hi], wi, bias=bi, activation="gelu_tanh")
        # every tile adds the products of 128 positions in the same order: the sums, and all that follows, are the same
        assert torch.equal(yi, y[lo:hi])
        dwi, dbi = torch.autograd.grad(yi, (wi, bi), g[lo:hi])
        assert torch.equal(dwi, dw[i])
        # values of at most 1.13 |g|; both sums take up to 40 additions in FP32 and are rounded at the end
        assert ((dbi - db[i]).abs() <= 2 * 42 * 2.0 ** -24 * 1.13 * g[lo:hi].double().abs().sum(0)).all()


def uneven(t, e, *key, front=0, behind=0):
    """Bounds of e groups, many of them empty or of one row."""
    r = np.random.default_rng([t, e, *key])
    share = np.exp2(r.integers(0, 7, e)) * (r.random(e) < 0.7)
    share[0], share[-1] = 0, 1                                             # the last group has rows, the first has none
    cuts = np.floor(np.cumsum(share) / share.sum() * (t - front - behind) + 1e-9).astype(np.int64)
    return np.concatenate([[0], cuts]) + front


@pytest.mark.parametrize("t,n,k,e", cases.MANY_GROUPS)
def test_many_groups(t, n, k, e):
    off = uneven(t, e, 20, front=2, behind=9)
    offsets = torch.from_numpy(off).cuda()
    a, w, bias = operand(t, k, 21), operand(e * n, k, 22, low=120), dense(e, n, torch.float32, 23)
    y = w.grouped_matmul(a, offsets, out_dtype=torch.bfloat16, bias=bias, activation="silu")
    assert not y[:2].any() and not y[-9:].any()
    r = np.random.default_rng([t, 24])
    some = [i for i in range(e) if off[i] < off[i + 1]]
    assert some[-1] == e - 1 and len(some) > e // 2
    for i in sorted({*r.choice(some, 25, replace=False), some[0], some[-1], *[j for j in some if 60 < j % 64 or j % 64 < 2][:12]}):
        rows = np.unique([off[i], off[i + 1] - 1, r.integers(off[i], off[i + 1])])
        vb = fp4.MXTensor(w.codes[i * n:(i + 1) * n], w.scales[i * n:(i + 1) * n], n, k).dequant().double()
        at = torch.from_numpy(rows).cuda()
        va = fp4.MXTensor(a.codes[at], a.scales[at], len(rows), k)
        va = fp4.MXTensor.from_canonical(va.codes, va.scales, k).dequant().double()
        z, ez = ref.with_bias(*sums(va, vb, k), f64(bias[i]))
        ref.check(y[at], *ref.out(z, ez, "silu", None, y.dtype), label=f"{t} {e} {i}")


@pytest.mark.parametrize("t,m,n,e", cases.MANY_GRADIENTS)
def test_weight_gradients_of_many_groups(t, m, n, e):
    off = uneven(t, e, 25, behind=5)
    offsets = torch.from_numpy(off).cuda()
    x, g = dense(t, n, torch.bfloat16, 26), dense(t, m, torch.bfloat16, 27)
    w = torch.zeros(e, m, n, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    (dw,) = torch.autograd.grad(fp4.mx_grouped_linear(x, w, offsets), w, g)
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo == hi:
            assert not dw[i].any()
            continue
        want, tol = ref.product(ref.values(g[lo:hi].T), ref.values(x[lo:hi].T), hi - lo)
        ref.check(dw[i], want, ref.rounded(want, tol, dw.dtype), f"{t} {e} {i}")
