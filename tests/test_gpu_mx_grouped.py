"""MXFP4 products of experts on the GPU against FP64: rows in groups of every kind and size, each kernel and tile, what belongs to
no group, the grouped quantisation bit for bit, the layer's gradients, streams and graphs."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import mx
from tests import mx_reference as ref
from tests.mx_epilogue_cases import GRADIENT_TILES, GROUPED_TILES
from tests.mx_reference import TYPES, dense, f64

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu

COMBOS = [(None, None, None, "bf16", "bf16"), ("silu", "bf16", "bf16", "packed", "f32"), ("gelu", "f32", None, "f16", "f16"),
          (None, None, "f32", "packed", "bf16"), ("gelu_tanh", "f16", "f32", "f32", "bf16"), ("relu", None, None, "packed", "f32")]


def bounds(t, e, *key, front=0, behind=0):
    """e + 1 bounds over t rows, groups of very different size, some empty."""
    r = np.random.default_rng([8, t, e, *key])
    share = np.exp2(r.integers(0, 6, e)) * (r.random(e) < 0.8)
    if not share.any():
        share[e // 2] = 1
    cuts = np.floor(np.cumsum(share) / share.sum() * (t - front - behind) + 1e-9).astype(np.int64)
    return np.concatenate([[0], cuts]) + front


def counted(values, t):
    """The bounds as the library counts them."""
    return np.maximum.accumulate(np.clip(np.asarray(values, np.int64), 0, t))


def grouped_product(va, vb, off, n, k):
    """(sums, their bound), zero for rows of no group."""
    z, ez = np.zeros((len(va), n)), np.zeros((len(va), n))
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            z[lo:hi], ez[lo:hi] = ref.product(va[lo:hi], vb[e * n:(e + 1) * n], k)
    return z, ez


def expert_of(off, t):
    """(expert of each row, whether it has one)."""
    e = np.searchsorted(off, np.arange(t), side="right") - 1
    inside = (np.arange(t) >= off[0]) & (np.arange(t) < off[-1])
    return np.clip(e, 0, len(off) - 2), inside


def forward(t, n, k, e, off, combo, *key, wide=False):
    name, bias, residual, x, o = combo
    w = fp4.MXTensor.quantize(dense(e * n, k, torch.float32, 1, *key, scale=0.1))
    a = dense(t, k, torch.bfloat16 if x == "packed" else TYPES[x], 2, *key)
    va, vb = ref.values(a), f64(w.dequant())
    if x == "packed":
        a = fp4.MXTensor.quantize(a)
    b = None if bias is None else dense(e, n, TYPES[bias], 3, *key)
    r = None if residual is None else dense(t, n, TYPES[residual], 4, *key)
    offsets = torch.from_numpy(np.asarray(off)).to(torch.int64 if wide else torch.int32).cuda()
    y = w.grouped_matmul(a, offsets, out_dtype=TYPES[o], bias=b, activation=name, residual=r)
    off = counted(off, t)
    expert, inside = expert_of(off, t)
    z, ez = grouped_product(va, vb, off, n, k)
    z, ez = ref.with_bias(z, ez, None if b is None else f64(b)[expert])
    want, tol = ref.out(z, ez, name, None if r is None else f64(r), TYPES[o])
    outside = np.zeros((t, n)) if r is None else f64(r)
    want[~inside] = outside[~inside]
    tol[~inside] = ref.HALF[TYPES[o]] * np.abs(want[~inside]) + ref.TINY[TYPES[o]]
    ref.check(y, want, tol, f"{t} {n} {k} {e} {combo}")
    return w, a, offsets, y, dict(bias=b, activation=name, residual=r), inside


@pytest.mark.parametrize("t,n,k,e", GROUPED_TILES)
def test_products(t, n, k, e):
    some = COMBOS if t * n * k < 10 ** 9 else [COMBOS[t % 6], COMBOS[(t + 1) % 6]]
    for c, combo in enumerate(some):
        front, behind = ((0, 0), (0, min(3, t - 1)), (min(2, t - 1), 0))[c % 3]
        forward(t, n, k, e, bounds(t, e, c, front=front, behind=behind), combo, c, wide=bool(c % 2))


@pytest.mark.parametrize("t,n,k,e", [(16, 70, 96, 5), (200, 130, 320, 5), (520, 1500, 96, 64), (2000, 2570, 96, 5)])
def test_groups_of_every_kind(t, n, k, e):
    cases = [[0] * e + [t], [0] + [t] * e, [0] * (e + 1), [t] * (e + 1), [0] * (e // 2 + 1) + [t] * (e - e // 2),   # one has all, none has any
             list(np.linspace(0, t, e + 1).astype(int)), [5] * e + [6], list(range(e + 1)), list(range(t - e, t + 1)),
             [0] + [1] * (e - 1) + [t]]
    if t >= 200:
        cases += [[0] + [min(t, 64 * i) for i in range(1, e + 1)], [0] + [min(t, 64 * i + 1) for i in range(1, e + 1)],
                  [0] + [min(t, 128 * i - 1) for i in range(1, e + 1)], [0] + [min(t, 17 * i) for i in range(1, e + 1)]]
    for c, off in enumerate(cases):
        forward(t, n, k, e, off, COMBOS[c % 6], 20, wide=bool(c % 2))


@pytest.mark.parametrize("t", [12, 300])
def test_bounds_that_make_no_sense_touch_nothing_else(t):
    """Decreasing, negative and far too large bounds count as documented; every row is some expert's or no one's."""
    n, k, e = 70, 96, 6
    big = 2 ** 40
    for c, off in enumerate(([0, 5, 3, 8, 2, 7, t], [-4, -1, 2, 2, t + 5, t + 9, 3], [t + 1] * 7, [-9] * 7, [4, 3, 2, 1, 0, -1, -2],
                             [3, big, 0, 1, 2, -big, 5], [0, t, 0, t, 0, t, 0])):
        if max(off) < 2 ** 31 and min(off) >= -2 ** 31:
            forward(t, n, k, e, off, COMBOS[c % 6], 30)
        forward(t, n, k, e, off, COMBOS[c % 6], 30, wide=True)


@pytest.mark.parametrize("e", [1, 2, 63, 64, 65, 127, 128, 129, 512])
def test_any_number_of_groups(e):
    for t in (9, 16, 17, 700):
        forward(t, 40, 64, e, bounds(t, e, behind=t // 9), COMBOS[1], 40, wide=bool(e % 2))


@pytest.mark.parametrize("t,n,k,e", [(13, 100, 96, 4), (150, 100, 96, 4), (600, 1500, 160, 64), (2000, 2570, 520, 5)])
def test_rows_of_no_group_are_left_alone(t, n, k, e):
    off = bounds(t, e, front=3, behind=4)
    w, a, offsets, want, kw, inside = forward(t, n, k, e, off, COMBOS[1], 50)
    for left, pad in ((0, 0), (1, 2)):
        wide = dense(t + 2, n + left + pad, torch.float32, 51)
        before = wide.clone()
        y = w.grouped_matmul(a, offsets, out=wide[1:-1, left:left + n], **kw)
        assert torch.equal(y[inside], want[inside])
        rest = torch.ones_like(wide, dtype=torch.bool)
        rest[1:-1, left:left + n][inside] = False
        assert torch.equal(wide[rest], before[rest])
    fp4.w4a4_grouped_matmul(t, n, k, a.codes, a.scales, w.codes, w.scales, offsets, wide[1:-1, 1:1 + n], fill=True, **kw)
    assert torch.equal(wide[1:-1, 1:1 + n], want)
    # the residual as the output
    y = kw["residual"].float()
    w.grouped_matmul(a, offsets, out=y, **(kw | {"residual": y}))
    assert torch.equal(y[inside], want[inside]) and torch.equal(y[~inside], kw["residual"].float()[~inside])
    x = torch.zeros(t, k, dtype=torch.bfloat16, device="cuda")
    y = torch.full((t, n), 7.0, device="cuda")
    fp4.w4a4_grouped_linear(t, n, k, x, w.codes, w.scales, offsets, y)
    assert not y[inside].any() and (y[~inside] == 7).all()


@pytest.mark.parametrize("t,n,k,e", [(12, 100, 96, 4), (150, 100, 96, 4), (700, 1500, 160, 64), (2000, 2570, 96, 5)])
def test_what_is_not_finite_stays_where_it_is(t, n, k, e):
    """NaN and infinities in rows of no expert, in weights of experts without rows, and in one row and one weight row."""
    off = bounds(t, e, 60, front=2, behind=3)
    x, wd = dense(t, k, torch.float32, 61), dense(e * n, k, torch.float32, 62)
    b = dense(e, n, torch.float32, 63)
    offsets = torch.from_numpy(off).cuda()
    want = fp4.MXTensor.quantize(wd).grouped_matmul(x, offsets, bias=b, activation="silu")
    _, inside = expert_of(off, t)
    x[~inside] = float("nan")
    for i in range(e):
        if off[i] == off[i + 1]:
            wd[i * n:(i + 1) * n] = float("inf")
            b[i] = float("nan")
    w = fp4.MXTensor.quantize(wd)
    assert torch.equal(w.grouped_matmul(x, offsets, bias=b, activation="silu"), want)
    row = int(off[0]) + (int(off[-1]) - int(off[0])) // 2
    x[row, 5] = float("nan")
    some = int(expert_of(off, t)[0][row])
    wd[some * n + 3] = float("inf")
    y = fp4.MXTensor.quantize(wd).grouped_matmul(x, offsets, bias=b, activation="silu")
    lo, hi = int(off[some]), int(off[some + 1])
    bad = torch.zeros_like(want, dtype=torch.bool)
    bad[row], bad[lo:hi, 3] = True, True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], want[~bad])


def test_past_32_bit_offsets():
    e, n, k = 9, 32_768, 32_768                                          # 4.8 GB of codes
    codes = torch.zeros(e * n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((e * n, k // 32), 120, dtype=torch.uint8, device="cuda")
    last = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    codes[-n:] = last
    w = fp4.MXTensor.from_canonical(codes, scales)
    for t in (3, 40):
        x = dense(t, k, torch.bfloat16, 64)
        off = torch.tensor([0] * e + [t], dtype=torch.int32, device="cuda")
        y = w.grouped_matmul(x, off)
        some = [0, 1, 777, n - 1]
        vb = mx.dequant(last[some].cpu().numpy(), scales[some].cpu().numpy())
        z, ez = ref.product(ref.values(x), vb, k)
        ref.check(y[:, some], *ref.out(z, ez, None, None, torch.float32))


def test_no_rows():
    w = fp4.MXTensor.quantize(dense(3 * 40, 64, torch.float32, 65))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert w.grouped_matmul(torch.empty(0, 64, device="cuda"), off, activation="gelu").shape == (0, 40)
    x, wd = torch.empty(0, 64, device="cuda", requires_grad=True), dense(3 * 40, 64, torch.float32, 66).reshape(3, 40, 64).requires_grad_()
    b = dense(3, 40, torch.float32, 67).requires_grad_()
    for name in (None, "silu"):
        y = fp4.mx_grouped_linear(x, wd, off, bias=b, activation=name)
        dx, dw, db = torch.autograd.grad(y, (x, wd, b), torch.empty(0, 40, device="cuda"))
        assert y.shape == (0, 40) and dx.shape == (0, 64) and not dw.any() and not db.any()


# ------------------------------------------------------------------------------------------- grouped quantisation

def quantize_grouped(x, off, e, rows=True, cols=True, z=None, name=None, db=None):
    """Through the C entry point: (rows codes, scales, columns' codes, scales, dbias), their memory full of 0xA5 before."""
    t, k = x.shape
    depth, nb = fp4.lib().fp4_grouped_depth(t, e), -(-k // 32)
    lds = (nb + 3) // 4 * 4
    q, s = (torch.full((t + 1, c), 0xA5, dtype=torch.uint8, device="cuda") for c in (16 * nb, lds))
    qt, st = (torch.full((k + 1, c), 0xA5, dtype=torch.uint8, device="cuda") for c in (depth // 2, depth // 32))
    a, at = fp4.Mx(q.data_ptr(), s.data_ptr(), 16 * nb, lds), fp4.Mx(qt.data_ptr(), st.data_ptr(), depth // 2, depth // 32)
    ty = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
    out = None if db is None else torch.full((e + 1, k), 7.0, dtype=db, device="cuda")
    ws = torch.empty(fp4.lib().fp4_grouped_sums_bytes(t, k, e), dtype=torch.uint8, device="cuda").fill_(255)
    act = [None, "relu", "silu", "gelu", "gelu_tanh"].index(name)
    grad = fp4.Gradient(None if z is None else z.data_ptr(), None if out is None else out.data_ptr(), 0 if z is None else z.stride(0), act,
                        0 if db is None else ty[db])
    groups = fp4.Groups(None if off is None else off.data_ptr(), e, 32)
    ref_ = ctypes.byref
    rc = fp4.lib().fp4_quantize_mxfp4_grouped(ty[x.dtype], t, k, x.data_ptr(), x.stride(0), ref_(groups), ref_(a) if rows else None,
                                              ref_(at) if cols else None, ref_(grad), ws.data_ptr(), ws.numel(),
                                              torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert (q[t] == 0xA5).all() and (s[t] == 0xA5).all() and (qt[k] == 0xA5).all() and (st[k] == 0xA5).all()
    assert out is None or (out[e] == 7).all()
    return q[:t].cpu().numpy(), s[:t].cpu().numpy(), qt[:k].cpu().numpy(), st[:k].cpu().numpy(), None if out is None else out[:e]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,k,e", [(1, 1, 1), (5, 33, 3), (300, 100, 4), (257, 130, 1), (700, 300, 40), (2050, 4100, 5), (3000, 70, 300)])
def test_quantize(dtype, t, k, e):
    x = dense(t, k + 3, TYPES[dtype], 70)[:, 1:1 + k]
    if t > 4 and k > 4:
        x[4, 2], x[3, 4] = float("inf"), float("nan")
    nb = -(-k // 32)
    alike = [None] if t % e == 0 else []
    for c, off in enumerate([bounds(t, e, 71, behind=t // 7), bounds(t, e, 72, front=t // 5)] + alike):
        offsets = None if off is None else torch.from_numpy(off).int().cuda()
        low = np.arange(e + 1) * (t // e) if off is None else off
        q, s, qt, st, _ = quantize_grouped(x, offsets, e, rows=c != 1, cols=True)
        x64 = f64(x)
        codes, scales = mx.quantize(x64)
        _, inside = expert_of(low, t)
        if c != 1:
            assert np.array_equal(q[inside], codes[inside]) and np.array_equal(s[inside][:, :nb], scales[inside]) and not s[inside][:, nb:].any()
            assert (q[~inside] == 0xA5).all() and (s[~inside] == 0xA5).all()
        else:
            assert (q == 0xA5).all() and (s == 0xA5).all()
        unit = 0
        for lo, hi in zip(low, low[1:]):
            units = -(-(hi - lo) // 256)
            if units:
                part = np.zeros((256 * units, k))
                part[:hi - lo] = x64[lo:hi]
                codes, scales = mx.quantize(part.T)
                assert np.array_equal(qt[:, 128 * unit:128 * (unit + units)], codes)
                assert np.array_equal(st[:, 8 * unit:8 * (unit + units)], scales)
            unit += units
        assert (qt[:, 128 * unit:] == 0xA5).all() and (st[:, 8 * unit:] == 0xA5).all()
    q, s, qt, st, _ = quantize_grouped(x, torch.from_numpy(bounds(t, e, 71)).int().cuda(), e, rows=True, cols=False)
    assert (qt == 0xA5).all() and (st == 0xA5).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", mx.ACTIVATIONS)
def test_quantize_a_gradient(dtype, name):
    """D = g f'(z): each value one that rounding at the border of D's tolerance allows, and the sums of g f'(z)."""
    t, k, e = 700, 330, 5
    off = bounds(t, e, 73, front=3, behind=9)
    g, z = dense(t, k, TYPES[dtype], 74), dense(t, k + 1, torch.float32, 75)[:, :k]
    z[5, :6] = torch.tensor([0.0, -0.0, 50.0, -50.0, 1e30, -1e30])
    _, inside = expert_of(off, t)
    z[~inside] = float("nan")                                              # not read into anything
    g[~inside] = float("inf")
    offsets = torch.from_numpy(off).int().cuda()
    for db in (torch.float32, TYPES[dtype], None):
        q, s, qt, st, sums = quantize_grouped(g, offsets, e, z=z, name=name, db=db)
        g64, z64 = np.where(inside[:, None], f64(g), 0), np.where(inside[:, None], f64(z), 0)
        if name is not None:
            z64 = np.clip(z64, -300, 300)                                   # f' is 0 or 1 from far below that on
        low, high = ref.gradient_interval(g64, z64, np.zeros_like(z64), name, TYPES[dtype])
        lo, hi = mx.quantize_interval(low, high)
        got = mx.dequant(q, s[:, :-(-k // 32)], k)
        assert ((lo <= got) & (got <= hi))[inside].all()
        assert np.count_nonzero(lo != hi) <= 4 + 0.01 * lo.size
        unit = 0
        for i, (a, b) in enumerate(zip(off, off[1:])):
            units = -(-(b - a) // 256)
            if units:
                lo, hi = mx.quantize_interval(low[a:b].T, high[a:b].T)
                got = mx.dequant(qt[:, 128 * unit:128 * (unit + units)], st[:, 8 * unit:8 * (unit + units)])
                assert ((lo <= got[:, :b - a]) & (got[:, :b - a] <= hi)).all() and not got[:, b - a:].any()
            unit += units
            if db is not None:
                want, tol = ref.bias_gradient(g64[a:b], z64[a:b], np.zeros((b - a, k)), name, db)
                ref.check(sums[i], want, tol, f"{i}")
    # the sums alone
    for db in (torch.float32, torch.bfloat16):
        q, s, qt, st, alone = quantize_grouped(g, offsets, e, rows=False, cols=False, z=z, name=name, db=db)
        assert torch.equal(alone, quantize_grouped(g, offsets, e, z=z, name=name, db=db)[4]) and (q == 0xA5).all() and (qt == 0xA5).all()


# ------------------------------------------------------------------------------------------------- the layer

def check_layer(t, n, k, off, name, bias, residual, x_type, w_type, *key, wide=False, share=0.01):
    e = len(off) - 1
    x, w = dense(t, k, x_type, 80, *key).requires_grad_(), dense(e * n, k, w_type, 81, *key, scale=0.1).reshape(e, n, k).requires_grad_()
    b = dense(e, n, w_type, 82, *key).requires_grad_() if bias else None
    r = dense(t, n, x_type, 83, *key).requires_grad_() if residual else None
    g = dense(t, n, x_type, 84, *key)
    offsets = torch.from_numpy(np.asarray(off)).to(torch.int64 if wide else torch.int32).cuda()
    y = fp4.mx_grouped_linear(x, w, offsets, bias=b, activation=name, residual=r)
    expert, inside = expert_of(off, t)
    label = f"{t} {n} {k} {e} {name} {x_type}"
    z, ez = grouped_product(ref.values(x), ref.values(w.reshape(e * n, k)), off, n, k)
    z, ez = ref.with_bias(z, ez, None if b is None else f64(b)[expert])
    want, tol = ref.out(z, ez, name, None if r is None else f64(r), x_type)
    want[~inside] = 0 if r is None else f64(r)[~inside]
    ref.check(y, want, tol, label)
    if r is None:
        assert not y[~inside].any()
    leaves = [v for v in (x, w, b, r) if v is not None]
    grads = torch.autograd.grad(y, leaves, g)
    assert [v.dtype for v in grads] == [v.dtype for v in leaves] and [v.shape for v in grads] == [v.shape for v in leaves]
    assert not grads[0][~inside].any()
    low, high = ref.gradient_interval(f64(g), z, ez, name, x_type)
    wide_of = 0
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo == hi:
            assert not grads[1][i].any() and (b is None or not grads[2][i].any())
            continue
        dlow, dhigh = low[lo:hi], high[lo:hi]
        want, tol = ref.interval_product(dlow, dhigh, ref.values(w[i].T), n)
        ref.check(grads[0][lo:hi], want, ref.rounded(want, tol, x_type), f"{label} dx {i}")
        want, tol = ref.interval_product(dlow.T, dhigh.T, ref.values(x[lo:hi].T), hi - lo)
        ref.check(grads[1][i], want, ref.rounded(want, tol, w_type), f"{label} dw {i}")
        if b is not None:
            ref.check(grads[2][i], *ref.bias_gradient(f64(g[lo:hi]), z[lo:hi], ez[lo:hi], name, w_type), f"{label} dbias {i}")
        a, c = mx.quantize_interval(dlow, dhigh)
        wide_of += np.count_nonzero(a != c)
    assert wide_of <= 4 + share * t * n
    if r is not None:
        assert torch.equal(grads[-1], g)


@pytest.mark.parametrize("t,n,k,e", [(1, 8, 32, 1), (5, 40, 33, 3), (16, 66, 70, 20), (40, 130, 64, 2), (300, 100, 200, 3), (1000, 264, 130, 7)])
@pytest.mark.parametrize("name", mx.ACTIVATIONS)
def test_layer(t, n, k, e, name):
    for i, (bias, residual) in enumerate(((True, True), (False, False), (True, False))):
        off = bounds(t, e, i, behind=min(i, t - 1), front=min(i // 2, t - 1))
        check_layer(t, n, k, off, name, bias, residual, (torch.bfloat16, torch.float32, torch.float16)[(i + t) % 3],
                    (torch.float32, torch.bfloat16)[i % 2], i, wide=bool(i % 2))


@pytest.mark.parametrize("t,n,k,e", GRADIENT_TILES)
def test_weight_gradients_in_every_tile(t, n, k, e):
    check_layer(t, n, k, bounds(t, e, 85, behind=1), "relu", True, False, torch.bfloat16, torch.bfloat16, 85, share=0.1)


def test_layer_is_its_experts_layers():
    """Each expert's slice through the dense layer: the same blocks, so the same values up to the order of FP32 sums."""
    t, n, k, e = 900, 200, 320, 6
    off = bounds(t, e, 86)
    x, w = dense(t, k, torch.float32, 87).requires_grad_(), dense(e * n, k, torch.float32, 88, scale=0.1).reshape(e, n, k).requires_grad_()
    g = dense(t, n, torch.float32, 89)
    got = fp4.mx_grouped_linear(x, w, torch.from_numpy(off).cuda())
    dx, dw = torch.autograd.grad(got, (x, w), g)
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo == hi:
            continue
        xi, wi = x[lo:hi].detach().requires_grad_(), w[i].detach().requires_grad_()
        y = fp4.mx_linear(xi, wi)
        dxi, dwi = torch.autograd.grad(y, (xi, wi), g[lo:hi])
        for a, b, p, q in ((got[lo:hi], y, xi, wi), (dx[lo:hi], dxi, g[lo:hi], wi.T), (dw[i], dwi, g[lo:hi].T, xi.T)):
            depth = p.shape[1]
            mag = ref.mm(np.abs(ref.values(p)), np.abs(ref.values(q)))
            ref.check(a, f64(b), 2 * mx.sum_bound(depth, mag) + 2.0 ** -23 * np.abs(f64(b)))


def test_layer_partial_gradients_and_twice():
    t, n, k, e = 60, 40, 64, 3
    x, w = dense(t, k, torch.bfloat16, 90), dense(e * n, k, torch.float32, 91).reshape(e, n, k)
    b, r, g = dense(e, n, torch.float32, 92), dense(t, n, torch.bfloat16, 93), dense(t, n, torch.bfloat16, 94)
    off = torch.tensor([2, 20, 20, 50], device="cuda")

    def run(which, name):
        leaf = {"x": x, "w": w, "bias": b, "residual": r}
        leaf = {i: v.clone().requires_grad_(i in which) for i, v in leaf.items()}
        y = fp4.mx_grouped_linear(leaf["x"].reshape(2, 30, k), leaf["w"], off, bias=leaf["bias"], activation=name, residual=leaf["residual"].reshape(2, 30, n))
        assert y.shape == (2, 30, n)
        return y, dict(zip(which, torch.autograd.grad(y, [leaf[i] for i in which], g.reshape(2, 30, n))))
    for name in (None, "gelu"):
        y, every = run(("x", "w", "bias", "residual"), name)
        for which in (("x",), ("w",), ("bias",), ("residual",), ("x", "bias"), ("w", "residual")):
            y1, some = run(which, name)
            assert torch.equal(y, y1) and all(torch.equal(some[i], every[i]) for i in which)
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = fp4.mx_grouped_linear(xl, wl, off, activation="silu")
    first = torch.autograd.grad(y, (xl, wl), g, retain_graph=True)
    for p, q in zip(torch.autograd.grad(y, (xl, wl), g.T.contiguous().T, retain_graph=True), first):
        assert torch.equal(p, q)
    once = torch.autograd.grad(y, (xl, wl), g, create_graph=True, retain_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        sum(v.float().sum() for v in once).backward()
    off.add_(0)                                                            # the bounds changed behind the graph's back
    with pytest.raises(RuntimeError, match="modified"):
        torch.autograd.grad(y, (xl, wl), g)


# ------------------------------------------------------------------------------------------- streams and graphs

def test_streams_and_threads():
    t, n, k, e = 300, 200, 512, 8
    w = fp4.MXTensor.quantize(dense(e * n, k, torch.bfloat16, 100))
    xt = dense(k, t, torch.bfloat16, 101)
    off = torch.from_numpy(bounds(t, e, 102, behind=5)).cuda()
    wide = torch.stack([off, off], 1)[:, 0]                                # bounds across memory are copied
    kw = dict(bias=dense(e, n, torch.float32, 103), activation="silu")
    want = w.grouped_matmul(xt.T, off, **kw)
    assert torch.equal(w.grouped_matmul(xt.T, wide, **kw), want)
    ws = torch.empty(fp4.w4a4_grouped_linear_workspace_bytes(t, n, k, e), dtype=torch.uint8, device="cuda").fill_(255)
    assert ws.numel() and torch.equal(w.grouped_matmul(xt.T, off, workspace=ws, **kw), want)
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        for _ in range(4):
            busy @ busy
        y = w.grouped_matmul(xt.T, wide, stream=given, **kw)
        side.synchronize()
        assert torch.equal(y.cpu(), want.cpu())
    bad = []

    def run(i):
        own = torch.cuda.Stream()
        with torch.cuda.stream(own):
            for _ in range(20):
                y = w.grouped_matmul(xt.T, off, **kw)
                own.synchronize()
                if not torch.equal(y, want):
                    bad.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(60)
    assert not bad


@pytest.mark.parametrize("t", [9, 16, 150, 1500])
def test_in_a_graph_whose_bounds_change(t):
    n, k, e = 200, 256, 6
    w = fp4.MXTensor.quantize(dense(e * n, k, torch.bfloat16, 110))
    x = dense(t, k, torch.bfloat16, 111)
    off = torch.from_numpy(bounds(t, e, 112)).cuda()
    call = lambda: w.grouped_matmul(x, off, activation="gelu", out_dtype=torch.bfloat16)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    for i in range(5):
        x.copy_(dense(t, k, torch.bfloat16, 113 + i))
        off.copy_(torch.from_numpy(bounds(t, e, 114, i, front=i % 2, behind=i)))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, call())
        torch.cuda.synchronize()


def test_training_step_in_a_graph_beside_an_eager_one():
    t, n, k, e = 400, 96, 128, 5
    x, g = dense(t, k, torch.bfloat16, 120).requires_grad_(), dense(t, n, torch.bfloat16, 121)
    w, b = dense(e * n, k, torch.float32, 122).reshape(e, n, k).requires_grad_(), dense(e, n, torch.float32, 123).requires_grad_()
    off = torch.from_numpy(bounds(t, e, 124)).cuda()

    def step():
        y = fp4.mx_grouped_linear(x, w, off, bias=b, activation="silu")
        return y, *torch.autograd.grad(y, (x, w, b), g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(), step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        with torch.no_grad():
            x.copy_(dense(t, k, torch.bfloat16, 125 + i))
        g.copy_(dense(t, n, torch.bfloat16, 126 + i))
        off.copy_(torch.from_numpy(bounds(t, e, 127, i, behind=2 * i)))
        graph.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in got]
        for p, q in zip(kept, step()):
            assert torch.equal(p, q)
        torch.cuda.synchronize()


def test_a_mixture_of_experts_together():
    """Tokens routed to two of five experts each, up with silu, down, weighted and added to the residual stream; for one token and for
    many, and a training step through both layers."""
    k, f, e, top = 128, 192, 5, 2
    wu, wd = dense(e * f, k, torch.float32, 130, scale=0.2).reshape(e, f, k), dense(e * k, f, torch.float32, 131, scale=0.2).reshape(e, k, f)
    up, down = fp4.MXTensor.quantize(wu), fp4.MXTensor.quantize(wd)
    for tokens in (1, 7, 300):
        x = dense(tokens, k, torch.bfloat16, 132)
        share, chosen = torch.softmax(dense(tokens, e, torch.float32, 133), 1).topk(top, 1)
        order = torch.argsort(chosen.reshape(-1), stable=True)
        off = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
        off[1:] = torch.bincount(chosen.reshape(-1), minlength=e).cumsum(0)
        rows = order // top
        h = up.grouped_matmul(x[rows], off, activation="silu", out_dtype=torch.bfloat16)
        y = down.grouped_matmul(h, off)
        mixed = x.float().index_add(0, rows, y * share.reshape(-1)[order][:, None])
        # token by token, from the same intermediate values
        vd, vh = f64(down.dequant()).reshape(e, k, f), ref.values(h)
        where = torch.empty_like(order)
        where[order] = torch.arange(order.numel(), device="cuda")
        want, tol = f64(x), np.zeros((tokens, k))
        for i in range(tokens):
            for j in range(top):
                row = int(where[i * top + j])
                z, ez = ref.product(vh[row:row + 1], vd[int(chosen[i, j])], f)
                s = float(share[i, j])
                want[i] += s * z[0]
                tol[i] += s * (ez[0] + 2.0 ** -22 * np.abs(z[0]))
        ref.check(mixed, want, tol + 2.0 ** -21 * np.abs(want) + 2.0 ** -22 * np.abs(f64(x)))
    xl, wul, wdl = x[rows].clone().requires_grad_(), wu.clone().requires_grad_(), wd.clone().requires_grad_()
    hl = fp4.mx_grouped_linear(xl, wul, off, activation="silu")
    g = dense(xl.shape[0], k, torch.bfloat16, 134)
    both = torch.autograd.grad(fp4.mx_grouped_linear(hl, wdl, off), (xl, wul, wdl), g)
    h2 = hl.detach().requires_grad_()
    dh, dwd = torch.autograd.grad(fp4.mx_grouped_linear(h2, wdl, off), (h2, wdl), g)
    dx, dwu = torch.autograd.grad(fp4.mx_grouped_linear(xl, wul, off, activation="silu"), (xl, wul), dh)
    for p, q in zip(both, (dx, dwu, dwd)):
        assert torch.equal(p, q)
