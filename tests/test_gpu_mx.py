"""MXFP4 on the GPU against the FP64 oracle: quantisation (bit for bit), its inverse, the products at sizes around
every tile, wave and block boundary, the dense-activation form, the trainable layer, streams, graphs and strides."""
import numpy as np
import pytest
import torch

from oracle import mx

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the smallest step


def rng(*key):
    return np.random.default_rng([20261206, *key])


def dense(m, k, dtype, *key, special=False):
    """Normal values with rows of very different size, zero blocks and, if asked, extreme and non-finite ones."""
    r = rng(m, k, *key)
    x = r.standard_normal((m, k)) * np.exp2(r.integers(-6, 7, (m, 1)))
    x[r.random((m, k)) < 0.01] = 0.0
    if k >= 64:
        x[:, 32:64] *= (r.random((m, 1)) < 0.7)
    t = torch.from_numpy(x).float()
    if special:
        info = torch.finfo(dtype)
        smallest = info.smallest_normal * info.eps
        t = t.to(dtype).float()
        flat = t.view(-1)
        for i, v in enumerate([info.max, -info.max, info.tiny, smallest, -smallest, 3 * smallest, -0.0, info.tiny * 6,
                               float("inf"), float("-inf"), float("nan")]):
            if flat.numel() > 97 * (i + 1):
                flat[97 * (i + 1)] = v
        if m > 2:
            t[2] = t[2].clamp(-1, 1) * smallest * 5          # a row of subnormals
            t[2][torch.isnan(t[2])] = 0
        if m > 3:
            t[3] = 0
    return t.to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check_operand(t, x64):
    codes, scales = mx.quantize(x64)
    assert np.array_equal(t.scales.cpu().numpy(), scales)
    assert np.array_equal(t.codes.cpu().numpy(), codes)


def close(y, ref, mag, k, label=""):
    """An output of the product against FP64: the sum's bound, then one rounding to the output's type."""
    tol = mx.sum_bound(k, mag)
    tol = tol + EPS[y.dtype] * (np.abs(ref) + tol) + TINY[y.dtype]
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), f"{label}: worst {np.max(err / tol)} of the tolerance"


# --------------------------------------------------------------------------------------------- quantisation

SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (2, 40), (3, 64), (5, 100), (31, 129), (32, 128), (33, 127), (64, 512),
          (127, 96), (128, 128), (129, 260), (130, 1000), (200, 1001), (1, 4096), (257, 2560)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("name", TYPES)
def test_quantize(name, m, k):
    x = dense(m, k, TYPES[name], special=True).cuda()
    rows, cols = fp4.MXTensor.quantize(x), fp4.MXTensor.quantize_t(x)
    both = fp4.MXTensor.quantize_both(x)
    torch.cuda.synchronize()
    x64 = f64(x)
    for t in (rows, both[0]):
        check_operand(t, x64)
    for t in (cols, both[1]):
        check_operand(t, x64.T)


@pytest.mark.parametrize("name", TYPES)
def test_quantize_every_pattern(name):
    # every bf16 / FP16 value (FP32: the bf16 ones with random low halves) as a block's one value, with a larger
    # neighbour that fixes the scale at several distances, and next to every midpoint of the grid
    bits = np.arange(65536, dtype=np.uint32)
    if name == "f32":
        v = torch.from_numpy(((bits << 16) | rng(7).integers(0, 65536, 65536).astype(np.uint32)).view(np.float32).copy())
    elif name == "bf16":
        v = torch.from_numpy(bits.astype(np.uint16).view(np.int16).copy()).view(torch.bfloat16)
    else:
        v = torch.from_numpy(bits.astype(np.uint16).view(np.float16).copy())
    x = torch.zeros(65536, 32, dtype=TYPES[name])
    x[:, 5] = v
    for shift in (1.0, 2.0, 6.5, 40.0):
        x[:, 17] = (v.float() * shift).to(TYPES[name])
        check_operand(fp4.MXTensor.quantize(x.cuda()), f64(x))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.98])
    x = torch.zeros(3 * mids.numel() * 2, 32)
    x[:, 0] = 4.0
    near = torch.cat([mids, mids * (1 - 2.0 ** -7), mids * (1 + 2.0 ** -7)])
    x[:, 9] = torch.cat([near, -near])
    x = x.to(TYPES[name])
    check_operand(fp4.MXTensor.quantize(x.cuda()), f64(x))
    check_operand(fp4.MXTensor.quantize_t(x.T.contiguous().cuda()), f64(x))


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_quantize_strided_rows(name, offset):
    base = dense(77, 300, TYPES[name], 1).cuda()
    x = base[:, offset:offset + 161]
    check_operand(fp4.MXTensor.quantize(x), f64(x))
    check_operand(fp4.MXTensor.quantize_t(x), f64(x).T)
    r, c = fp4.MXTensor.quantize_both(base.T)                 # a transposed view is copied
    check_operand(r, f64(base).T)
    check_operand(c, f64(base))


def test_quantize_leaves_the_rest_alone():
    x = dense(37, 75, torch.bfloat16, 2).cuda()
    q = torch.full((40, 64), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((40, 8), 0xA5, dtype=torch.uint8, device="cuda")
    qt = torch.full((80, 48), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.full((80, 8), 0xA5, dtype=torch.uint8, device="cuda")
    fp4.fp4_quantize_mxfp4(37, 75, x, q[:37, :48], s[:37, :3], qt[:75, :32], st[:75, :2])
    torch.cuda.synchronize()
    codes, scales = mx.quantize(f64(x))
    assert np.array_equal(q[:37, :48].cpu().numpy(), codes) and np.array_equal(s[:37, :3].cpu().numpy(), scales)
    assert (q[37:] == 0xA5).all() and (q[:, 48:] == 0xA5).all() and (s[37:] == 0xA5).all() and (s[:, 4:] == 0xA5).all()
    codes, scales = mx.quantize(f64(x).T)
    assert np.array_equal(qt[:75, :32].cpu().numpy(), codes) and np.array_equal(st[:75, :2].cpu().numpy(), scales)
    assert (qt[75:] == 0xA5).all() and (qt[:, 32:] == 0xA5).all() and (st[75:] == 0xA5).all() and (st[:, 4:] == 0xA5).all()


def test_quantize_past_32_bit_offsets():
    m, k = 70_001, 32_768                                     # 4.6 GB of bf16, 2.3e9 elements
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    tail = dense(300, k, torch.bfloat16, 4).cuda()
    x[-300:] = tail
    r, c = fp4.MXTensor.quantize_both(x)
    want = fp4.MXTensor.quantize(tail)
    assert torch.equal(r.codes[-300:], want.codes) and torch.equal(r.scales[-300:], want.scales)
    r2 = fp4.MXTensor.quantize(x)
    assert torch.equal(r2.codes, r.codes) and torch.equal(r2.scales, r.scales)
    first = (m - 300) // 32 * 32
    part = fp4.MXTensor.quantize_t(x[first:].contiguous())
    assert torch.equal(c.codes[:, first // 2:], part.codes) and torch.equal(c.scales[:, first // 32:], part.scales)
    back = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    fp4.fp4_dequant_mxfp4(m, k, r.codes, r.scales, back)
    assert torch.equal(back[-300:], want.dequant(torch.bfloat16)) and not back[0].any()


def test_quantize_no_rows():
    x = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    t = fp4.MXTensor.quantize(x)
    assert t.rows == 0 and t.dequant().shape == (0, 100)


# --------------------------------------------------------------------------------------------------- inverse

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dequant_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).reshape(256, 16, 16).reshape(256 * 16, 16)
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).reshape(-1, 1)
    t = fp4.MXTensor.from_canonical(codes.cuda(), scales.cuda())
    want = torch.from_numpy(mx.dequant(codes.numpy(), scales.numpy())).to(torch.float32)
    got = t.dequant(dtype).float().cpu()
    # FP32 and bf16 hold every value; 4 and 6 times 2^127 become infinity (scale 254)
    assert torch.equal(torch.nan_to_num(got, nan=1.25), torch.nan_to_num(want, nan=1.25))


@pytest.mark.parametrize("k", [1, 7, 8, 9, 33, 100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dequant_ragged_and_strided(k, dtype):
    x = dense(21, k, torch.float32, 5).cuda()
    t = fp4.MXTensor.quantize(x)
    out = torch.full((25, k + 3), 7.0, dtype=dtype, device="cuda")
    fp4.fp4_dequant_mxfp4(21, k, t.codes, t.scales, out[:21, 1:k + 1])
    codes, scales = mx.quantize(f64(x))
    assert np.array_equal(f64(out[:21, 1:k + 1]), mx.dequant(codes, scales, k))
    assert (out[21:] == 7).all() and (out[:, 0] == 7).all() and (out[:, k + 1:] == 7).all()


# --------------------------------------------------------------------------------------------------- product

PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 15, 64), (2, 17, 33), (3, 40, 100), (1, 64, 4096), (5, 33, 160), (15, 16, 256), (16, 48, 288),
            (17, 31, 96), (32, 64, 384), (33, 70, 1000), (48, 100, 512), (64, 128, 2080), (64, 1, 257), (65, 1, 32), (65, 129, 96),
            (100, 257, 256), (127, 128, 288), (128, 127, 512), (129, 130, 544), (150, 150, 768), (128, 128, 800), (200, 333, 1056),
            (257, 511, 1280), (300, 260, 5000), (70, 90, 9728)]


def operands(m, n, k, *key):
    a, b = dense(m, k, torch.float32, 10, *key), dense(n, k, torch.float32, 11, *key)
    return mx.quantize(f64(a)), mx.quantize(f64(b))


def upload(op, k):
    return fp4.MXTensor.from_canonical(torch.from_numpy(op[0]).cuda(), torch.from_numpy(op[1]).cuda(), k)


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k):
    a, b = operands(m, n, k)
    ref, mag = mx.product(mx.dequant(*a, k), mx.dequant(*b, k))
    ta, tb = upload(a, k), upload(b, k)
    for dtype in TYPES.values():
        scale = 1.0
        y = tb.matmul(ta, out_dtype=dtype)
        if dtype == torch.float16:
            ok = np.abs(ref) < 60000
            assert ok.mean() > 0.5
            y, r, g = y[torch.from_numpy(ok).cuda()], ref[ok], mag[ok]
        else:
            r, g = ref, mag
        close(y, r * scale, g, k, f"{m}x{n}x{k} {dtype}")
    # without a workspace K is not split
    y = torch.empty(m, n, device="cuda")
    fp4.w4a4_matmul(m, n, k, ta.codes, ta.scales, tb.codes, tb.scales, y,
                    workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    close(y, ref, mag, k, "no workspace")


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 320), (4095, 4097, 544), (4100, 5000, 32), (2048, 9728, 2560),
                                   (4096, 4608, 4096), (4090, 4601, 4100)])
def test_product_large_tiles(m, n, k):
    a = dense(m, k, torch.bfloat16, 12).cuda()
    b = dense(n, k, torch.bfloat16, 13).cuda()
    ta, tb = fp4.MXTensor.quantize(a), fp4.MXTensor.quantize(b)
    y = tb.matmul(ta, out_dtype=torch.float32)
    yb = tb.matmul(ta, out_dtype=torch.bfloat16)
    a64, b64 = ta.dequant().double(), tb.dequant().double()
    ref, mag = a64 @ b64.T, a64.abs() @ b64.abs().T
    tol = torch.from_numpy(np.array(mx.sum_bound(k, 1.0))).cuda() * mag
    assert ((y.double() - ref).abs() <= tol + 2.0 ** -24 * (ref.abs() + tol)).all()
    assert ((yb.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -134).all()
    assert torch.equal(y, tb.matmul(ta))                       # the same bits every time


@pytest.mark.parametrize("m,n,k", [(1, 300, 1024), (9, 64, 512), (64, 64, 512), (130, 260, 1024), (4096, 4096, 512)])
def test_product_of_small_whole_numbers_is_exact(m, n, k):
    r = rng(m, n, k)
    a = torch.from_numpy(r.choice([-6.0, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (m, k))).float().cuda()
    b = torch.from_numpy(r.choice([-6.0, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (n, k))).float().cuda()
    a[:, 0::32] = 4.0                                          # every scale is 2^0
    b[:, 0::32] = 4.0
    y = fp4.MXTensor.quantize(b).matmul(fp4.MXTensor.quantize(a))
    assert torch.equal(y.double(), a.double() @ b.double().T)


@pytest.mark.parametrize("m", [1, 40, 130])
def test_product_one_hot_and_identity(m):
    n, k = 140, 1000
    b = dense(n, k, torch.bfloat16, 14).cuda()
    tb = fp4.MXTensor.quantize(b)
    at = rng(m).integers(0, k, m)
    a = torch.zeros(m, k)
    a[torch.arange(m), torch.from_numpy(at)] = 1.0
    y = tb.matmul(fp4.MXTensor.quantize(a.cuda()))
    assert torch.equal(y, tb.dequant()[:, torch.from_numpy(at).cuda()].T)


@pytest.mark.parametrize("m", [2, 40, 130, 300])
def test_product_nan_and_infinite_values(m):
    n, k = 140, 700
    a, b = dense(m, k, torch.bfloat16, 15).cuda(), dense(n, k, torch.bfloat16, 16).cuda()
    clean = fp4.MXTensor.quantize(b).matmul(fp4.MXTensor.quantize(a))
    a[1, 699], b[137, 3] = float("nan"), float("inf")
    y = fp4.MXTensor.quantize(b).matmul(fp4.MXTensor.quantize(a))
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[1], bad[:, 137] = True, True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])
    yl = fp4.MXTensor.quantize(b).matmul(a)                    # dense activations
    assert torch.equal(torch.isnan(yl), bad)


@pytest.mark.parametrize("m", [3, 40, 150])
def test_product_far_scales(m):
    # block scales over the whole range of a byte: sums that overflow, vanish, or fit
    n, k = 130, 96
    r = rng(m, 5)
    for sa, sb in ((250, 5), (254, 0), (127, 127), (200, 180), (30, 60)):
        a = r.integers(0, 256, (m, 48), dtype=np.uint8), np.full((m, 3), sa, np.uint8)
        b = r.integers(0, 256, (n, 48), dtype=np.uint8), np.full((n, 3), sb, np.uint8)
        y = f64(upload(b, k).matmul(upload(a, k)))
        ref, mag = mx.product(mx.dequant(*a), mx.dequant(*b))
        if sa + sb - 254 + 12 > 127:
            # an FP32 sum: a partial sum past the range is an infinity of its own sign, which no later product takes
            # back (a product here reaches 36 2^126 by itself), so neither the sign nor inf against NaN is fixed by
            # the exact sum; that the result is not a finite number is
            big = np.abs(ref) >= 2.0 ** 128
            assert big.any() and not np.isfinite(y[big]).any()
        elif sa + sb - 254 < -170:
            assert (y == 0).all()
        else:
            assert (np.abs(y - ref) <= mx.sum_bound(k, mag) + 2.0 ** -149).all()


@pytest.mark.parametrize("m", [1, 20, 64, 130, 300])
@pytest.mark.parametrize("dtype", list(TYPES.values()))
def test_product_strides_and_bounds(m, dtype):
    # operands inside larger buffers whose surroundings are NaN blocks, an output with a stride and an odd offset
    n, k = 77, 416
    a, b = operands(m, n, k, 3)
    nb = k // 32
    held = []
    for codes, scales in (a, b):
        q = torch.full((codes.shape[0] + 2, codes.shape[1] + 64), 0x77, dtype=torch.uint8, device="cuda")
        s = torch.full((codes.shape[0] + 2, nb + 11), 255, dtype=torch.uint8, device="cuda")   # 24 bytes apart
        q[1:-1, 16:-48] = torch.from_numpy(codes).cuda()
        s[1:-1, 4:4 + nb] = torch.from_numpy(scales).cuda()
        held.append((q[1:-1, 16:-48], s[1:-1, 4:4 + nb]))
    y = torch.full((m + 1, n + 6), 7.0, dtype=dtype, device="cuda")
    (aq, a_s), (bq, bs) = held
    fp4.w4a4_matmul(m, n, k, aq, a_s, bq, bs, y[:m, 3:n + 3])
    ref, mag = mx.product(mx.dequant(*a), mx.dequant(*b))
    ok = np.abs(ref) < (60000 if dtype == torch.float16 else np.inf)
    got = y[:m, 3:n + 3]
    close(got[torch.from_numpy(ok).cuda()], ref[ok], mag[ok], k)
    assert (y[m:] == 7).all() and (y[:, :3] == 7).all() and (y[:, n + 3:] == 7).all()


def test_from_canonical_copies_what_is_not_aligned():
    m, n, k = 20, 50, 160                                     # 5 scale bytes a row: not a multiple of 4
    a, b = operands(m, n, k, 6)
    buf = torch.zeros(50 * 5 + 1, dtype=torch.uint8, device="cuda")
    buf[1:] = torch.from_numpy(b[1]).cuda().reshape(-1)
    odd = torch.zeros(50 * 80 + 8, dtype=torch.uint8, device="cuda")
    odd[8:] = torch.from_numpy(b[0]).cuda().reshape(-1)
    tb = fp4.MXTensor.from_canonical(odd[8:].view(50, 80), buf[1:].view(50, 5))
    ref, mag = mx.product(mx.dequant(*a), mx.dequant(*b))
    close(tb.matmul(upload(a, k)), ref, mag, k)


def test_product_past_32_bit_offsets():
    m, n = 66_000, 40_000                                      # 2.6e9 outputs
    a, b = dense(m, 32, torch.bfloat16, 20).cuda(), dense(n, 32, torch.bfloat16, 21).cuda()
    ta, tb = fp4.MXTensor.quantize(a), fp4.MXTensor.quantize(b)
    y = tb.matmul(ta, out_dtype=torch.bfloat16)
    for r in (slice(0, 70), slice(53_600, 53_800), slice(m - 70, m)):
        part = fp4.MXTensor(ta.codes[r], ta.scales[r], r.stop - r.start, 32)
        assert torch.equal(y[r], tb.matmul(part, out_dtype=torch.bfloat16))
    # weights past 2^31 bytes with one row of activations
    n, k = 270_000, 16_384                                     # 2.2e9 bytes of codes
    big = fp4.MXTensor.empty(n, k)
    big.codes.zero_()
    big.scales.fill_(127)
    tail = fp4.MXTensor.quantize(dense(100, k, torch.bfloat16, 22).cuda())
    big.codes[-100:], big.scales[-100:] = tail.codes, tail.scales
    for m in (1, 70):
        x = fp4.MXTensor.quantize(dense(m, k, torch.bfloat16, 23).cuda())
        y = big.matmul(x)
        assert not y[:, :-100].any()
        ref, mag = mx.product(f64(x.dequant()), f64(tail.dequant()))
        close(y[:, -100:], ref, mag, k)


def test_product_no_rows():
    b = fp4.MXTensor.quantize(dense(20, 64, torch.bfloat16, 24).cuda())
    assert b.matmul(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 20)
    assert b.matmul(fp4.MXTensor.empty(0, 64)).shape == (0, 20)


# ------------------------------------------------------------------------------------------ dense activations

@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 40, 33), (1, 512, 4096), (2, 33, 100), (7, 64, 511), (15, 100, 1000), (16, 48, 2560),
                                   (17, 40, 96), (33, 70, 1001), (64, 128, 513), (65, 90, 300), (129, 257, 777), (300, 260, 2000)])
@pytest.mark.parametrize("name", TYPES)
def test_linear(name, m, n, k):
    x = dense(m, k, TYPES[name], 30).cuda()
    b = mx.quantize(f64(dense(n, k, torch.float32, 31)))
    tb = upload(b, k)
    xq = mx.quantize(f64(x))
    ref, mag = mx.product(mx.dequant(*xq, k), mx.dequant(*b, k))
    for dtype in (torch.float32, torch.bfloat16):
        close(tb.matmul(x, out_dtype=dtype), ref, mag, k, f"{m}x{n}x{k}")
    wide = torch.zeros(m, k + 5, dtype=x.dtype, device="cuda")
    wide[:, 1:k + 1] = x
    assert torch.equal(tb.matmul(wide[:, 1:k + 1]), tb.matmul(x))


# ---------------------------------------------------------------------------------------------------- training

def layer_reference(x, w, g):
    """The layer's y, dx, dw in FP64 and the magnitudes behind them."""
    q = lambda t: mx.dequant(*mx.quantize(t), t.shape[1])  # noqa: E731
    y = mx.product(q(x), q(w))
    dx = mx.product(q(g), q(w.T))
    dw = mx.product(q(g.T), q(x.T))
    return y, dx, dw


@pytest.mark.parametrize("m,n,k", [(1, 32, 32), (5, 40, 64), (33, 70, 100), (64, 96, 160), (100, 130, 300), (257, 200, 333)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f16", "f16")])
def test_layer_and_its_gradients(m, n, k, types):
    x = dense(m, k, TYPES[types[0]], 40).mul(0.01).cuda().requires_grad_()
    w = dense(n, k, TYPES[types[1]], 41).mul(0.01).cuda().requires_grad_()
    g = dense(m, n, TYPES[types[0]], 42).mul(0.01).cuda()
    y = fp4.mx_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), g)
    assert y.dtype == x.dtype and dx.dtype == x.dtype and dw.dtype == w.dtype
    ry, rdx, rdw = layer_reference(f64(x), f64(w), f64(g))
    close(y, *ry, k, "y")
    close(dx, *rdx, n, "dx")
    close(dw, *rdw, m, "dw")


def test_layer_gradients_against_differences():
    # The layer stands for y = x w^T, which is linear in x and in w: differences of <g, x w^T> are exact gradients of
    # it. A block's values move by at most a quarter of its largest magnitude in quantisation (2 scales of the 4 to 8
    # that it measures), so the products' difference is bounded by the moves of their factors.
    m, n, k = 96, 80, 128
    x, w, g = dense(m, k, torch.float32, 50), dense(n, k, torch.float32, 51), dense(m, n, torch.float32, 52)
    xc, wc = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    dx, dw = torch.autograd.grad(fp4.mx_linear(xc, wc), (xc, wc), g.cuda())
    x, w, g = x.double().numpy(), w.double().numpy(), g.double().numpy()

    def move(t):
        nb = mx.blocks(t.shape[1])
        pad = np.zeros((t.shape[0], nb * 32))
        pad[:, :t.shape[1]] = np.abs(t)
        return np.repeat(pad.reshape(t.shape[0], nb, 32).max(axis=2) / 4, 32, axis=1)[:, :t.shape[1]]

    r = rng(53)
    for grad, at, left, right in ((dx, x, g, w.T), (dw, w, g.T, x.T)):
        v = r.standard_normal(at.shape)
        f = (lambda t: float((g * (t @ w.T)).sum())) if at is x else (lambda t: float((g * (x @ t.T)).sum()))
        h = 0.5
        slope = (f(at + h * v) - f(at - h * v)) / (2 * h)
        ml, mr = move(left), move(right)
        bound = (np.abs(left) @ mr.T + ml @ np.abs(right).T + ml @ mr.T)
        diff = float((f64(grad) * v).sum())
        assert abs(diff - slope) <= float((bound * np.abs(v)).sum())
        # and far closer than that bound as a direction: the rounding errors do not line up
        exact = left @ right.T
        cos = float((f64(grad) * exact).sum() / np.linalg.norm(f64(grad)) / np.linalg.norm(exact))
        assert cos > 0.95


def test_layer_partial_gradients_shapes_and_no_rows():
    x = dense(24, 64, torch.bfloat16, 60).cuda()
    w = dense(40, 64, torch.bfloat16, 61).cuda()
    g = dense(24, 40, torch.bfloat16, 62).cuda()
    x3 = x.reshape(2, 3, 4, 64)
    xg, wg = x3.clone().requires_grad_(), w.clone().requires_grad_()
    y = fp4.mx_linear(xg, wg)
    assert y.shape == (2, 3, 4, 40)
    dx, dw = torch.autograd.grad(y, (xg, wg), g.reshape(2, 3, 4, 40))
    only_x = torch.autograd.grad(fp4.mx_linear(xg, w), xg, g.reshape(2, 3, 4, 40))[0]
    only_w = torch.autograd.grad(fp4.mx_linear(x3, wg), wg, g.reshape(2, 3, 4, 40))[0]
    assert torch.equal(only_x, dx) and torch.equal(only_w, dw)
    # an expanded gradient, as sum() gives
    (da,) = torch.autograd.grad(fp4.mx_linear(xg, w).sum(), xg)
    (db,) = torch.autograd.grad(fp4.mx_linear(xg, w), xg, torch.ones(2, 3, 4, 40, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(da, db)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = fp4.mx_linear(e, wg)
    dx, dw = torch.autograd.grad(y, (e, wg), torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 40) and dx.shape == (0, 64) and not dw.any()


def test_layer_twice_and_in_place():
    x = dense(24, 64, torch.bfloat16, 63).cuda().requires_grad_()
    w = dense(40, 64, torch.float32, 64).cuda().requires_grad_()
    g = dense(24, 40, torch.bfloat16, 65).cuda()
    want = torch.autograd.grad(fp4.mx_linear(x, w), (x, w), g)
    y = fp4.mx_linear(x, w)
    for a, b in zip(torch.autograd.grad(y, (x, w), g, retain_graph=True), want):
        assert torch.equal(a, b)
    for a, b in zip(torch.autograd.grad(y, (x, w), g), want):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError):                          # freed
        torch.autograd.grad(y, (x, w), g)
    y = fp4.mx_linear(x, w).mul_(2.0)
    for a, b in zip(torch.autograd.grad(y, (x, w), g / 2), want):
        assert torch.equal(a, b)
    # differentiable once: a second derivative is an error, not a zero
    dx, dw = torch.autograd.grad(fp4.mx_linear(x, w), (x, w), g, create_graph=True)
    assert torch.equal(dx, want[0])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dx.float().sum() + dw.sum(), x)
    with pytest.raises(RuntimeError, match="once"):
        (dx.float().sum() + dw.sum()).backward()
    (dw,) = torch.autograd.grad(fp4.mx_linear(x.detach(), w), w, g, create_graph=True)
    assert torch.equal(dw, want[1])
    with torch.no_grad():
        assert not fp4.mx_linear(x, w).requires_grad


def test_a_few_layers_together():
    # prefill through a gated pair of projections in both forms: quantised once for two products, or dense
    m, k, f = 70, 256, 300
    x = dense(m, k, torch.bfloat16, 70).mul(0.1).cuda()
    gate, up, down = (fp4.MXTensor.quantize(dense(a, b, torch.float32, 71 + i).cuda())
                      for i, (a, b) in enumerate(((f, k), (f, k), (k, f))))
    xq = fp4.MXTensor.quantize(x)
    ga, ua = gate.matmul(xq, out_dtype=torch.bfloat16), up.matmul(xq, out_dtype=torch.bfloat16)
    assert torch.equal(ga, gate.matmul(x, out_dtype=torch.bfloat16))
    h = (torch.sigmoid(ga.float()) * ua.float()).to(torch.bfloat16)
    y = down.matmul(h)
    ref, mag = mx.product(mx.dequant(*mx.quantize(f64(h)), f), f64(down.dequant()))
    close(y, ref, mag, f)
    # one token of it at a time gives the same rows to the order of the sums
    for r in (0, 13, 69):
        close(down.matmul(h[r:r + 1]), ref[r:r + 1], mag[r:r + 1], f)


# ------------------------------------------------------------------------------------------- streams and graphs

def test_other_stream_and_given_workspace():
    m, n, k = 150, 200, 4096
    x, b = dense(m, k, torch.bfloat16, 80).cuda(), fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 81).cuda())
    want = b.matmul(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        y = torch.empty(m, n, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        b.matmul(x, out=y, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
    ws = torch.empty(fp4.w4a4_linear_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda").fill_(255)
    assert torch.equal(b.matmul(x, workspace=ws), want)


@pytest.mark.parametrize("raw", [False, True])
def test_given_stream_orders_copies_and_outputs(raw):
    """Inputs that have to be copied first, on a stream that does not wait for the busy current one."""
    m, n, k = 200, 160, 1024
    xt = dense(k, m, torch.bfloat16, 100).cuda()
    w = dense(n, k, torch.bfloat16, 101).cuda()
    b = fp4.MXTensor.quantize(w)
    want = b.matmul(xt.t().contiguous())
    both = fp4.MXTensor.quantize_both(xt.t().contiguous())
    wide = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(4):
            wide @ wide
        s = side.cuda_stream if raw else side
        y = b.matmul(xt.t(), stream=s)
        qr, qc = fp4.MXTensor.quantize_both(xt.t(), stream=s)
        d = qr.dequant(stream=s)
        side.synchronize()
        assert torch.cuda.current_stream() != side
        got = [t.cpu() for t in (y, qr.codes, qr.scales, qc.codes, qc.scales, d)]
        for g, e in zip(got, (want, both[0].codes, both[0].scales, both[1].codes, both[1].scales, both[0].dequant())):
            assert torch.equal(g, e.cpu())


def test_two_streams_at_once():
    """Calls with workspaces of their own, interleaved on two streams from two threads."""
    import threading
    m, n, k = 40, 200, 8192
    b = fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 102).cuda())
    assert fp4.w4a4_linear_workspace_bytes(m, n, k) > 0
    xs = [dense(m, k, torch.bfloat16, 103 + i).cuda() for i in range(2)]
    want = [b.matmul(x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(20):
                y = b.matmul(xs[i])
                side.synchronize()
                if not torch.equal(y, want[i]):
                    bad.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad


def test_layer_with_broadcast_and_transposed_gradients():
    """Gradients that arrive without memory of their own (a sum's) or across the rows, inputs shared by two layers."""
    n, k = 96, 160
    x3 = dense(5 * 14, k, torch.float32, 105).reshape(5, 14, k).transpose(0, 1).cuda()
    w = dense(n, k, torch.float32, 106).cuda().requires_grad_()
    x = x3.detach().requires_grad_()
    y = fp4.mx_linear(x, w)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    ex, ew = torch.autograd.grad(fp4.mx_linear(x, w), (x, w), torch.ones(14, 5, n, device="cuda"))
    assert torch.equal(dx, ex) and torch.equal(dw, ew)
    g = dense(n, 70, torch.float32, 107).cuda().t().reshape(14, 5, n)
    gt = g.contiguous().transpose(0, 1).contiguous().transpose(0, 1)
    dx, dw = torch.autograd.grad(fp4.mx_linear(x, w), (x, w), gt)
    ex, ew = torch.autograd.grad(fp4.mx_linear(x, w), (x, w), g.contiguous())
    assert torch.equal(dx, ex) and torch.equal(dw, ew)
    # the same weights twice: the gradients of the two uses add
    (d2,) = torch.autograd.grad([fp4.mx_linear(x, w), fp4.mx_linear(x, w)], w, [g, g])
    assert torch.equal(d2, ew + ew)


@pytest.mark.parametrize("m,n,k", [(12, 4100, 2080), (16, 2560, 4096), (9, 4130, 2592), (1, 4099, 4640), (3, 2049, 9760)])
def test_few_rows_of_wide_weights(m, n, k):
    """Few rows through the workspace as well as quantised inside the product, workgroups of eight and of ten waves,
    waves with several lines of K."""
    x = dense(m, k, torch.bfloat16, 120).cuda()
    b = fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 121).cuda())
    a = fp4.MXTensor.quantize(x)
    ref, mag = mx.product(f64(a.dequant()), f64(b.dequant()))
    close(b.matmul(x), ref, mag, k, "dense")
    close(b.matmul(a, out_dtype=torch.bfloat16), ref, mag, k, "MXFP4")
    ws = torch.full((fp4.w4a4_linear_workspace_bytes(m, n, k),), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((m + 2, n), 7.0, device="cuda")
    b.matmul(x, out=y[1:-1], workspace=ws)
    close(y[1:-1], ref, mag, k, "workspace")
    assert (y[0] == 7).all() and (y[-1] == 7).all()


@pytest.mark.parametrize("m", [1, 9, 40, 150])
def test_linear_in_a_graph(m):
    n, k = 200, 2048
    b = fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 82).cuda())
    x = dense(m, k, torch.bfloat16, 83).cuda()
    b.matmul(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.matmul(x)
    for i in range(4):
        x.copy_(dense(m, k, torch.bfloat16, 84 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, b.matmul(x))
        torch.cuda.synchronize()


def test_training_step_in_a_graph_beside_an_eager_one():
    m, n, k = 130, 96, 512
    x = dense(m, k, torch.bfloat16, 90).cuda()
    w = dense(n, k, torch.float32, 91).cuda().requires_grad_()
    g = dense(m, n, torch.bfloat16, 92).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(fp4.mx_linear(x, w), w, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fp4.mx_linear(x, w)
        (dw,) = torch.autograd.grad(y, w, g)
    for i in range(4):
        x.copy_(dense(m, k, torch.bfloat16, 93 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), dw.clone()
        ye = fp4.mx_linear(x, w)
        (de,) = torch.autograd.grad(ye, w, g)
        assert torch.equal(got[0], ye) and torch.equal(got[1], de)
        torch.cuda.synchronize()
