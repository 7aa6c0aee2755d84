"""MXFP4 products with bias, activation and residual on the GPU against FP64: every kernel and tile, types, strides, special
values, streams and graphs, and the layer's gradients against the formulas' and against differences."""
import itertools
import threading

import numpy as np
import pytest
import torch

from oracle import mx
from tests import mx_reference as ref
from tests.mx_reference import TYPES, dense, f64

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu

# few rows; tiles of 64, K in parts, 128, streams of 128, 256, columns behind whole rounds; edges of every kind
SIZES = [(1, 33, 100), (2, 64, 32), (9, 200, 4096), (16, 1030, 330), (17, 40, 64), (70, 130, 513), (40, 100, 9600), (64, 256, 2048), (300, 520, 1024),
         (257, 1000, 40), (1000, 2560, 1056), (1999, 2111, 1100), (4090, 4096, 300), (4100, 4099, 517), (8190, 8200, 288)]
COMBOS = [(None, "bf16", "bf16", "bf16", "bf16"), ("silu", None, None, "bf16", "bf16"), ("gelu", "f32", None, "packed", "f16"),
          ("gelu_tanh", None, "f32", "f16", "f32"), ("relu", "f16", "f16", "packed", "bf16"), (None, None, "f32", "packed", "f32"),
          ("silu", "bf16", "bf16", "f32", "f32"), ("gelu", "bf16", "f32", "bf16", "bf16")]


def operands(m, n, k, x, *key):
    """(activations in the form wanted, weights, their values)."""
    w = fp4.MXTensor.quantize(dense(n, k, torch.float32, 1, *key, scale=0.1))
    a = dense(m, k, torch.bfloat16 if x == "packed" else TYPES[x], 2, *key)
    va, vb = ref.values(a), f64(w.dequant())
    return fp4.MXTensor.quantize(a) if x == "packed" else a, w, va, vb


@pytest.mark.parametrize("m,n,k", SIZES)
def test_products(m, n, k):
    some = COMBOS if m * n < 10 ** 6 else COMBOS[m % 4::4]
    for c, (name, bias, residual, x, o) in enumerate(some):
        a, w, va, vb = operands(m, n, k, x, c)
        b = None if bias is None else dense(1, n, TYPES[bias], 3, c)[0]
        r = None if residual is None else dense(m, n, TYPES[residual], 4, c)
        y = w.matmul(a, out_dtype=TYPES[o], bias=b, activation=name, residual=r)
        z, ez = ref.product(va, vb, k)
        z, ez = ref.with_bias(z, ez, None if b is None else f64(b))
        ref.check(y, *ref.out(z, ez, name, None if r is None else f64(r), TYPES[o]), label=f"{m} {n} {k} {some[c]}")


@pytest.mark.parametrize("m,n,k", [(5, 70, 96), (40, 100, 9600), (130, 200, 320), (1000, 2050, 544), (4100, 4100, 288)])
@pytest.mark.parametrize("o", ["bf16", "f32"])
def test_residual_in_place_and_strided(m, n, k, o):
    a, w, va, vb = operands(m, n, k, "packed", 10)
    b = dense(1, 2 * n, torch.float32, 11)[0, ::2]                         # a bias across memory
    z, ez = ref.with_bias(*ref.product(va, vb, k), f64(b))
    for left, pad in ((0, 0), (3, 5), (8, 8)):
        wide = dense(m + 2, n + left + pad, TYPES[o], 12)
        before = wide.clone()
        r = f64(wide[1:-1, left:left + n])
        got = w.matmul(a, out=wide[1:-1, left:left + n], bias=b, activation="silu", residual=wide[1:-1, left:left + n])
        assert got.data_ptr() == wide[1:-1, left:left + n].data_ptr()
        ref.check(got, *ref.out(z, ez, "silu", r, TYPES[o]), label=f"{left}")
        rest = torch.ones_like(wide, dtype=torch.bool)
        rest[1:-1, left:left + n] = False
        assert torch.equal(wide[rest], before[rest])
    # a residual whose rows lie across memory, is copied; one that is expanded is too
    r = dense(n, m, torch.bfloat16, 13).T
    ref.check(w.matmul(a, out_dtype=TYPES[o], bias=b, residual=r), *ref.out(z, ez, None, f64(r), TYPES[o]))
    r = dense(1, n, torch.bfloat16, 14).expand(m, n)
    ref.check(w.matmul(a, out_dtype=TYPES[o], bias=b, residual=r), *ref.out(z, ez, None, f64(r), TYPES[o]))
    with pytest.raises(ValueError, match="residual"):
        y = torch.zeros(m, n, dtype=torch.float16, device="cuda")
        w.matmul(a, out=y, residual=y.view(torch.bfloat16))                # the output read as another type


def test_negated_views():
    m, n, k = 20, 40, 64
    a, w, va, vb = operands(m, n, k, "packed", 15)
    b, r = torch._neg_view(dense(1, n, torch.float32, 16)[0]), torch._neg_view(dense(m, n, torch.float32, 17))
    assert b.is_neg() and r.is_neg()
    z, ez = ref.with_bias(*ref.product(va, vb, k), f64(b))
    ref.check(w.matmul(a, bias=b, residual=r), *ref.out(z, ez, None, f64(r), torch.float32))
    with pytest.raises(ValueError, match="negated"):
        fp4.w4a4_matmul(m, n, k, a.codes, a.scales, w.codes, w.scales, torch.empty(m, n, device="cuda"), residual=r)


@pytest.mark.parametrize("m", [3, 40, 130])
@pytest.mark.parametrize("name", mx.ACTIVATIONS)
def test_every_size_of_a_sum(m, name):
    """Sums from the smallest to past FP32's range, and what is not finite, through the bias, the product being zero."""
    special = [0.0, -0.0, 1e-45, 1e-38, -1e-38, 1e-10, 3e38, -3e38, float("inf"), float("-inf"), float("nan")]
    grid = np.concatenate([np.linspace(-20, 20, 401), [-100, -90, -60, 60, 90, 100, 1e4, -1e4, 1e20, -1e20], special])
    n, k = grid.size, 64
    w = fp4.MXTensor.quantize(torch.zeros(n, k, device="cuda"))
    a = fp4.MXTensor.quantize(dense(m, k, torch.bfloat16, 20))
    b = torch.from_numpy(grid).float().cuda()
    y = f64(w.matmul(a, bias=b, activation=name))
    z = f64(b)
    with np.errstate(all="ignore"):
        finite = np.isfinite(z)
        want, tol = ref.out(np.where(finite, z, 0), np.zeros(n), name, None, torch.float32)
    assert (np.abs(y - want) <= tol)[:, finite].all(), np.nonzero(~(np.abs(y - want) <= tol)[:, finite])
    inf, minus, nan = y[:, -3], y[:, -2], y[:, -1]
    assert (inf == np.inf).all() and np.isnan(nan).all()
    if name is None:
        assert (minus == -np.inf).all()
    elif name in ("relu", "gelu"):
        assert (minus == 0).all()
    else:
        assert np.isnan(minus).all()
    # an output type's overflow, and a weight row that is NaN
    y = w.matmul(a, bias=b.clamp(max=1e5), activation=name, out_dtype=torch.float16)
    assert torch.isinf(y[:, -5]).all() if name != "relu" else True
    scales = w.scales.clone()
    scales[7] = 255
    y = fp4.MXTensor.from_canonical(w.codes, scales, k).matmul(a, bias=torch.ones(n, device="cuda"), activation=name)
    assert torch.isnan(y[:, 7]).all() and torch.isfinite(y[:, :7]).all() and torch.isfinite(y[:, 8:]).all()


def test_no_rows_and_repeatable():
    w = fp4.MXTensor.quantize(dense(100, 96, torch.float32, 30))
    y = w.matmul(torch.empty(0, 96, device="cuda"), bias=torch.zeros(100, device="cuda"), residual=torch.empty(0, 100, device="cuda"), activation="gelu")
    assert y.shape == (0, 100)
    for m, n, k in ((9, 4096, 4096), (64, 300, 9600), (4100, 4100, 544)):
        a, w, _, _ = operands(m, n, k, "bf16", 31)
        r = dense(m, n, torch.bfloat16, 32)
        first = w.matmul(a, activation="gelu", residual=r)
        for _ in range(3):
            assert torch.equal(first, w.matmul(a, activation="gelu", residual=r))


def test_past_32_bit_offsets():
    m, n, k = 40_003, 60_001, 64                                          # 2.4e9 outputs
    a, w = dense(m, k, torch.bfloat16, 33), dense(n, k, torch.bfloat16, 34)
    r = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 35_792, 35_793, m - 1]
    r[rows] = dense(len(rows), n, torch.bfloat16, 35)
    b = dense(1, n, torch.bfloat16, 36)[0]
    keep = r[rows].clone()
    y = fp4.MXTensor.quantize(w).matmul(a, out=r, bias=b, activation="relu", residual=r)
    z, ez = ref.with_bias(*ref.product(ref.values(a[rows]), ref.values(w), k), f64(b))
    ref.check(y[rows], *ref.out(z, ez, "relu", f64(keep), torch.bfloat16))


# ------------------------------------------------------------------------------------------- streams and graphs

def test_streams_workspaces_and_threads():
    m, n, k = 40, 200, 8192
    a, w, _, _ = operands(m, n, k, "bf16", 40)
    b, rt = dense(1, n, torch.float32, 41)[0], dense(n, m, torch.bfloat16, 42)
    kw = dict(bias=b, activation="gelu")
    want = w.matmul(a, residual=rt.T, **kw)
    ws = torch.empty(fp4.w4a4_linear_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda").fill_(255)
    assert ws.numel() > 0 and torch.equal(w.matmul(a, residual=rt.T, workspace=ws, **kw), want)
    # K not split for want of room: the same to the order of the sums
    small = torch.empty(m * k // 2 + m * k // 32 + 512, dtype=torch.uint8, device="cuda")
    va, vb = ref.values(a), f64(w.dequant())
    z, ez = ref.with_bias(*ref.product(va, vb, k), f64(b))
    ref.check(w.matmul(a, residual=rt.T, workspace=small, **kw), *ref.out(z, ez, "gelu", f64(rt).T, torch.float32))
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        for _ in range(4):
            busy @ busy
        y = w.matmul(a, residual=rt.T, stream=given, **kw)                 # copies the residual, on the stream
        side.synchronize()
        assert torch.equal(y.cpu(), want.cpu())
    bad = []

    def run(i):
        own = torch.cuda.Stream()
        with torch.cuda.stream(own):
            for _ in range(20):
                y = w.matmul(a, residual=rt.T, **kw)
                own.synchronize()
                if not torch.equal(y, want):
                    bad.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad


@pytest.mark.parametrize("m", [1, 9, 40, 150, 1000])
def test_in_a_graph(m):
    n, k = 200, 2048
    a, w, _, _ = operands(m, n, k, "bf16", 50)
    b, r = dense(1, n, torch.bfloat16, 51)[0], dense(m, n, torch.bfloat16, 52)
    call = lambda: w.matmul(a, bias=b, activation="silu", residual=r, out_dtype=torch.bfloat16)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    for i in range(4):
        a.copy_(dense(m, k, torch.bfloat16, 53 + i))
        r.copy_(dense(m, n, torch.bfloat16, 54 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, call())
        torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------------- the layer

def check_layer(m, n, k, name, bias, residual, x_type, w_type, *key, share=0.01):
    x, w = dense(m, k, x_type, 60, *key).requires_grad_(), dense(n, k, w_type, 61, *key, scale=0.1).requires_grad_()
    b = dense(1, n, w_type, 62, *key)[0].requires_grad_() if bias else None
    r = dense(m, n, x_type, 63, *key).requires_grad_() if residual else None
    g = dense(m, n, x_type, 64, *key)
    y = fp4.mx_linear(x, w, bias=b, activation=name, residual=r)
    assert y.dtype == x_type and y.shape == (m, n)
    z, ez = ref.with_bias(*ref.product(ref.values(x), ref.values(w), k), None if b is None else f64(b))
    label = f"{m} {n} {k} {name} {x_type}"
    ref.check(y, *ref.out(z, ez, name, None if r is None else f64(r), x_type), label=label)
    leaves = [t for t in (x, w, b, r) if t is not None]
    grads = torch.autograd.grad(y, leaves, g)
    assert [t.dtype for t in grads] == [t.dtype for t in leaves] and [t.shape for t in grads] == [t.shape for t in leaves]
    low, high = ref.gradient_interval(f64(g), z, ez, name, x_type)
    want, tol = ref.interval_product(low, high, ref.values(w.T), n)
    ref.check(grads[0], want, ref.rounded(want, tol, x_type), label + " dx")
    want, tol = ref.interval_product(low.T, high.T, ref.values(x.T), m)
    ref.check(grads[1], want, ref.rounded(want, tol, w_type), label + " dw")
    # few of D's values may lie within reach of a border (a handful of a small matrix, more where the worst case of a deep sum
    # is far from what happens): the interval says something
    lo, hi = mx.quantize_interval(low, high)
    assert np.count_nonzero(hi > lo) <= 4 + share * lo.size, label
    if b is not None:
        ref.check(grads[2], *ref.bias_gradient(f64(g), z, ez, name, w_type), label + " dbias")
    if r is not None:
        assert torch.equal(grads[-1], g)


@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (5, 40, 33), (31, 130, 64), (33, 64, 100), (257, 200, 130), (300, 1030, 96), (1000, 776, 520)])
@pytest.mark.parametrize("name", mx.ACTIVATIONS)
def test_layer(m, n, k, name):
    for i, (bias, residual) in enumerate(((True, True), (False, False), (True, False), (False, True))):
        if name is None and not bias and not residual:
            continue
        x_type = (torch.bfloat16, torch.float32, torch.float16, torch.bfloat16)[(i + m) % 4]
        check_layer(m, n, k, name, bias, residual, x_type, (torch.float32, torch.bfloat16)[i % 2], i)


@pytest.mark.parametrize("m,n,k,name", [(4100, 4099, 1030, "gelu"), (4099, 2050, 2570, "silu")])
def test_layer_in_large_tiles(m, n, k, name):
    check_layer(m, n, k, name, True, True, torch.bfloat16, torch.bfloat16, 9, share=0.1)


def test_gradients_are_differences():
    """Where every operand is a value that its 4 bits hold, along either axis, the gradients are those of the dense function,
    and central differences of it (relu, whose sums stay away from 0; a difference is exact up to FP64's rounding)."""
    m, n, k = 24, 40, 64
    r = np.random.default_rng(7)
    x, w, g = (torch.from_numpy(r.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 3.0], s)).float().cuda() for s in ((m, k), (n, k), (m, n)))
    for t in (x, w, g):
        t[:, 0] = 3.0                                                      # every block's scale is 2^-1 or so, along its rows
        t[0] = 3.0                                                         # and its columns
    x, w = x.requires_grad_(), w.requires_grad_()
    b = torch.from_numpy(r.standard_normal(n)).float().cuda().requires_grad_()
    got = torch.autograd.grad(fp4.mx_linear(x, w, bias=b, activation="relu"), (x, w, b), g)

    def loss(x, w, b):
        return (np.maximum(x @ w.T + b, 0) * f64(g)).sum()
    at = [f64(t) for t in (x, w, b)]
    z = at[0] @ at[1].T + at[2]
    assert np.array_equal(ref.values(x), at[0]) and np.array_equal(ref.values(w.T), at[1].T) and np.array_equal(ref.values(g.T), f64(g).T)
    h = np.abs(z).min() / 8
    assert h > 1e-6
    for which, grad in enumerate(got):
        for _ in range(40):
            i = tuple(r.integers(0, s) for s in at[which].shape)
            up, down = [t.copy() for t in at], [t.copy() for t in at]
            up[which][i] += h
            down[which][i] -= h
            d = (loss(*up) - loss(*down)) / (2 * h)
            # FP64's rounding of two losses of up to 1e5, over 2 h; FP32's of the sum of the gradient, of up to 40 values of 9
            assert abs(d - grad[i].item()) <= 1e5 * 2.0 ** -50 / h + 2.0 ** -23 * 40 * 360
    # and the smooth ones' bias gradients against differences of the library's own forward pass in FP32
    for name in ("silu", "gelu", "gelu_tanh"):
        f = lambda b: (fp4.mx_linear(x, w, bias=b, activation=name).double() * g.double()).sum().item()  # noqa: B023, E731
        (db,) = torch.autograd.grad(fp4.mx_linear(x, w, bias=b, activation=name), b, g)
        h, size = 2.0 ** -6, 2.0 ** 9                                      # y is below 2^9, good to 2^-14 of itself at most
        for i in (0, 7, n - 1):
            e = torch.zeros_like(b)
            e[i] = h
            d = (f(b.detach() + e) - f(b.detach() - e)) / (2 * h)
            # h^2 / 6 of a third derivative below 2, for m values of g up to 3; FP32 rounding of m values of y over 2 h
            assert abs(d - db[i].item()) <= m * 3 * (h * h / 3 + 2 * size * 2.0 ** -22 / (2 * h))


def test_layer_partial_gradients_shapes_and_no_rows():
    x, w, b, r, g = (dense(*s, t, 70 + i) for i, (s, t) in enumerate((((24, 64), torch.bfloat16), ((40, 64), torch.float32), ((1, 40), torch.float32),
                                                                     ((24, 40), torch.bfloat16), ((24, 40), torch.bfloat16))))
    b = b[0]
    leaves = {"x": x.reshape(2, 3, 4, 64), "w": w, "bias": b, "residual": r.reshape(2, 3, 4, 40)}
    g = g.reshape(2, 3, 4, 40)

    def run(which, name="gelu"):
        t = {k: v.clone().requires_grad_(k in which) for k, v in leaves.items()}
        y = fp4.mx_linear(t["x"], t["w"], bias=t["bias"], activation=name, residual=t["residual"])
        return y, dict(zip(which, torch.autograd.grad(y, [t[k] for k in which], g)))
    for name in ("gelu", None):
        y, all_of = run(("x", "w", "bias", "residual"), name)
        assert y.shape == (2, 3, 4, 40)
        for size in (1, 2, 3):
            for which in itertools.combinations(("x", "w", "bias", "residual"), size):
                got = run(which, name)
                assert torch.equal(got[0], y)
                for k, v in got[1].items():
                    assert torch.equal(v, all_of[k]), (which, k)
    with torch.no_grad():
        t = {k: v.clone().requires_grad_() for k, v in leaves.items()}
        assert not fp4.mx_linear(t["x"], t["w"], bias=t["bias"], activation="silu").requires_grad
    e, wg, bg = torch.empty(0, 64, device="cuda", requires_grad=True), w.clone().requires_grad_(), b.clone().requires_grad_()
    y = fp4.mx_linear(e, wg, bias=bg, activation="silu")
    dx, dw, db = torch.autograd.grad(y, (e, wg, bg), torch.empty(0, 40, device="cuda"))
    assert y.shape == (0, 40) and dx.shape == (0, 64) and not dw.any() and not db.any()
    # without anything behind the product it is the layer as it was
    assert torch.equal(fp4.mx_linear(x, w), fp4.mx_linear(x, w, bias=None, activation=None, residual=None))


def test_layer_twice_broadcast_and_shared():
    m, n, k = 70, 96, 160
    x, w = dense(m, k, torch.float32, 80).requires_grad_(), dense(n, k, torch.float32, 81).requires_grad_()
    b, r = dense(1, n, torch.float32, 82)[0].requires_grad_(), dense(m, n, torch.float32, 83).requires_grad_()
    f = lambda: fp4.mx_linear(x, w, bias=b, activation="gelu_tanh", residual=r)  # noqa: E731
    g = dense(m, n, torch.float32, 84)
    want = torch.autograd.grad(f(), (x, w, b, r), g)
    y = f()
    for _ in range(2):
        for p, q in zip(torch.autograd.grad(y, (x, w, b, r), g, retain_graph=True), want):
            assert torch.equal(p, q)
    for p, q in zip(torch.autograd.grad(f(), (x, w, b, r), dense(m, n, torch.float32, 84).T.contiguous().T), want):
        assert torch.equal(p, q)
    ones = torch.autograd.grad(f(), (x, w, b, r), torch.ones_like(g))
    for p, q in zip(torch.autograd.grad(f().sum(), (x, w, b, r)), ones):   # a gradient without memory of its own
        assert torch.equal(p, q)
    (d2,) = torch.autograd.grad([f(), f()], b, [g, g])
    assert torch.equal(d2, want[2] + want[2])
    once = torch.autograd.grad(f(), (x, b), g, create_graph=True)
    assert torch.equal(once[0], want[0])
    with pytest.raises(RuntimeError, match="once"):
        sum(t.sum() for t in once).backward()
    # the residual as the input itself: both gradients arrive
    s = dense(n, n, torch.float32, 85).requires_grad_()
    h = dense(m, n, torch.float32, 86).requires_grad_()
    (dh,) = torch.autograd.grad(fp4.mx_linear(h, s, residual=h), h, g)
    (dx,) = torch.autograd.grad(fp4.mx_linear(h, s), h, g)
    assert torch.equal(dh, dx + g)
    # a graph that saved the output notices that it is written over
    y = f().exp()
    with torch.no_grad():
        w4 = fp4.MXTensor.quantize(w.detach())
        w4.matmul(x.detach(), out=y, activation="relu")
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


def test_training_step_in_a_graph_beside_an_eager_one():
    m, n, k = 300, 96, 512
    x, w = dense(m, k, torch.bfloat16, 90), dense(n, k, torch.float32, 91).requires_grad_()
    b, g = dense(1, n, torch.float32, 92)[0].requires_grad_(), dense(m, n, torch.bfloat16, 93)

    def step():
        y = fp4.mx_linear(x, w, bias=b, activation="silu")
        return y, *torch.autograd.grad(y, (w, b), g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(), step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(dense(m, k, torch.bfloat16, 94 + i))
        g.copy_(dense(m, n, torch.bfloat16, 95 + i))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for p, q in zip(kept, step()):
            assert torch.equal(p, q)
        torch.cuda.synchronize()


def test_a_feed_forward_block_together():
    """Up with gelu, down onto the residual stream: token by token and at once, and its training step."""
    m, k, f = 70, 256, 640
    x = dense(m, k, torch.bfloat16, 96)
    wu, wd = dense(f, k, torch.float32, 97, scale=0.1), dense(k, f, torch.float32, 98, scale=0.1)
    bu, bd = dense(1, f, torch.float32, 99)[0], dense(1, k, torch.float32, 100)[0]
    up, down = fp4.MXTensor.quantize(wu), fp4.MXTensor.quantize(wd)
    h = up.matmul(x, bias=bu, activation="gelu", out_dtype=torch.bfloat16)
    y = down.matmul(h, bias=bd, residual=x, out_dtype=torch.bfloat16)
    z, ez = ref.with_bias(*ref.product(ref.values(h), ref.values(wd), f), f64(bd))
    ref.check(y, *ref.out(z, ez, None, f64(x), torch.bfloat16))
    for r in (0, 33, 69):
        ref.check(down.matmul(h[r:r + 1], bias=bd, residual=x[r:r + 1], out_dtype=torch.bfloat16),
                  *ref.out(z[r:r + 1], ez[r:r + 1], None, f64(x)[r:r + 1], torch.bfloat16))
    leaves = [t.clone().requires_grad_() for t in (x, wu, bu, wd, bd)]
    xl, wul, bul, wdl, bdl = leaves
    yl = fp4.mx_linear(fp4.mx_linear(xl, wul, bias=bul, activation="gelu"), wdl, bias=bdl, residual=xl)
    g = dense(m, k, torch.bfloat16, 101)
    grads = torch.autograd.grad(yl, leaves, g)
    # the lower layer's gradient is what the upper layer's is made of
    hl = fp4.mx_linear(x, wu, bias=bu, activation="gelu").requires_grad_()
    dh, dwd, dbd = torch.autograd.grad(fp4.mx_linear(hl, wdl, bias=bdl, residual=x), (hl, wdl, bdl), g)
    dx, dwu, dbu = torch.autograd.grad(fp4.mx_linear(xl, wul, bias=bul, activation="gelu"), (xl, wul, bul), dh)
    for p, q in zip(grads, (dx + g, dwu, dbu, dwd, dbd)):
        assert torch.equal(p, q)
