"""MXFP4 on the GPU: what the calls do to the memory, streams and gradients around them."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
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


def test_written_tensors_count_as_changed():
    """Autograd refuses to go back through a saved tensor that a call wrote over, as it does for torch's own writes."""
    m, n, k = 20, 48, 64
    x = dense(m, k, torch.bfloat16, 210).cuda()
    b = fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 211).cuda())
    a = fp4.MXTensor.quantize(x)
    scale = torch.ones(n, device="cuda", requires_grad=True)
    for write in (lambda y: b.matmul(x, out=y), lambda y: b.matmul(a, out=y),
                  lambda y: fp4.w4a4_linear(m, n, k, x, b.codes, b.scales, y),
                  lambda y: fp4.w4a4_matmul(m, n, k, a.codes, a.scales, b.codes, b.scales, y)):
        y = torch.randn(m, n, device="cuda")
        loss = (y * scale).sum()
        write(y)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    out = torch.empty(m, k, device="cuda")
    q, s, qt, st = (torch.zeros(*shape, dtype=torch.uint8, device="cuda") for shape in ((m, 32), (m, 4), (k, 16), (k, 4)))
    before = [t._version for t in (out, q, s, qt, st)]
    fp4.fp4_dequant_mxfp4(m, k, a.codes, a.scales, out)
    fp4.fp4_quantize_mxfp4(m, k, x, q, s[:, :2], qt, st[:, :1])
    assert all(t._version > v for t, v in zip((out, q, s, qt, st), before))
    # the inputs are not written
    assert x._version == a.codes._version == b.scales._version == 0
    with torch.inference_mode():
        y = torch.empty(m, n, device="cuda")
    assert torch.equal(b.matmul(x, out=y), b.matmul(x))        # no version to count


def test_lazily_negated_views():
    """The imaginary part of a conjugate is a view whose memory holds the other sign."""
    z = torch.complex(dense(70, 96, torch.float32, 220), dense(70, 96, torch.float32, 221)).cuda()
    for part in (z.conj().imag, z[:, :1].conj().imag, z[0].conj().imag, torch._neg_view(z.real.contiguous())):
        assert part.is_neg()
        plain = part.resolve_neg().contiguous()
        got, want = fp4.MXTensor.quantize_both(part), fp4.MXTensor.quantize_both(plain)
        for g, w in zip(got, want):
            assert torch.equal(g.codes, w.codes) and torch.equal(g.scales, w.scales)
        b = fp4.MXTensor.quantize(dense(40, part.shape[-1], torch.float32, 222).cuda())
        if part.dim() == 2:
            assert torch.equal(b.matmul(part), b.matmul(plain))
        w = dense(40, part.shape[-1], torch.float32, 223).cuda()
        assert torch.equal(fp4.mx_linear(part, w), fp4.mx_linear(plain, w))
    x, w = dense(70, 96, torch.float32, 224).cuda().requires_grad_(), dense(96, 96, torch.float32, 225).cuda().requires_grad_()
    g = torch._neg_view(z.real.contiguous())
    for got, want in zip(torch.autograd.grad(fp4.mx_linear(x, w), (x, w), g), torch.autograd.grad(fp4.mx_linear(x, w), (x, w), g.resolve_neg())):
        assert torch.equal(got, want)
    q, s = torch.empty(70, 48, dtype=torch.uint8, device="cuda"), torch.empty(70, 4, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="negated"):
        fp4.fp4_quantize_mxfp4(70, 96, g, q, s[:, :3])
    with pytest.raises(ValueError, match="negated"):
        fp4.fp4_dequant_mxfp4(70, 96, q, s[:, :3], g)


def test_a_stream_of_another_gpu_is_refused():
    x = dense(20, 64, torch.bfloat16, 230).cuda()
    b = fp4.MXTensor.quantize(dense(40, 64, torch.bfloat16, 231).cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = b.matmul(x)

    class Elsewhere:                                           # as a torch stream of a second GPU looks
        cuda_stream, device = side.cuda_stream, torch.device("cuda", x.device.index + 1)

    y, out = torch.empty(20, 40, device="cuda"), torch.empty(20, 64, device="cuda")
    for call in (lambda s: fp4.MXTensor.quantize_both(x, stream=s), lambda s: b.matmul(x, stream=s), lambda s: b.matmul(b, stream=s),
                 lambda s: b.dequant(stream=s), lambda s: fp4.w4a4_linear(20, 40, 64, x, b.codes, b.scales, y, stream=s),
                 lambda s: fp4.w4a4_matmul(20, 40, 64, b.codes[:20], b.scales[:20], b.codes, b.scales, y, stream=s),
                 lambda s: fp4.fp4_dequant_mxfp4(20, 64, b.codes[:20], b.scales[:20], out, stream=s),
                 lambda s: fp4.fp4_quantize_mxfp4(20, 64, x, b.codes[:20], b.scales[:20], stream=s)):
        with pytest.raises(ValueError, match="stream belongs"):
            call(Elsewhere())
    class Bare:                                                # a handle and nothing else
        cuda_stream = side.cuda_stream

    for s in (side, side.cuda_stream, Bare(), torch.cuda.current_stream(), 0):
        got = b.matmul(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("m", [3, 40, 150])
@pytest.mark.parametrize("e", [-120, -126, -130, -138, -147])
def test_sums_below_the_normal_range(m, e):
    """Scales whose product is 2^e: every product is a multiple of 2^(e - 2), at least FP32's smallest step, and the sum of
    96 of them, at most 36 2^e each, has under 24 bits above it. So every sum, subnormal or not, is exact."""
    n, k, sa = 130, 96, 60
    r = np.random.default_rng([m, -e])
    a = r.integers(0, 256, (m, 48), dtype=np.uint8), np.full((m, 3), sa, np.uint8)
    b = r.integers(0, 256, (n, 48), dtype=np.uint8), np.full((n, 3), 254 + e - sa, np.uint8)
    ta, tb = (fp4.MXTensor.from_canonical(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), k) for q, s in (a, b))
    ref, _ = mx.product(mx.dequant(*a), mx.dequant(*b))
    assert (np.abs(ref) < 2.0 ** -126).any() or e == -120
    assert np.array_equal(tb.matmul(ta).cpu().double().numpy(), ref)


@pytest.mark.parametrize("what", ["dense", "MXFP4", "layer"])
def test_two_threads_on_two_streams(what):
    """Each thread's calls are counted and its errors are raised here."""
    m, n, k, times = 40, 200, 8192, 20
    w = dense(n, k, torch.bfloat16, 240).cuda()
    b = fp4.MXTensor.quantize(w)
    assert fp4.w4a4_matmul_workspace_bytes(m, n, k) > 0
    xs = [dense(m, k, torch.bfloat16, 241 + i).cuda() for i in range(2)]

    def call(x):
        if what == "layer":
            x, v = x.detach().requires_grad_(), w.detach().requires_grad_()
            y = fp4.mx_linear(x, v)
            return y.detach(), *torch.autograd.grad(y, (x, v), torch.ones_like(y))
        return (b.matmul(x if what == "dense" else fp4.MXTensor.quantize(x)),)

    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    done = [0, 0]

    def run(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(times):
                got = call(xs[i])
                side.synchronize()
                done[i] += all(torch.equal(g, v) for g, v in zip(got, want[i]))

    with ThreadPoolExecutor(2) as pool:
        for f in [pool.submit(run, i) for i in range(2)]:
            f.result(timeout=60)
    assert done == [times, times]


def test_layer_in_inference_mode():
    x, w = dense(24, 64, torch.bfloat16, 250).cuda(), dense(40, 64, torch.float32, 251).cuda().requires_grad_()
    want = fp4.mx_linear(x, w.detach())
    with torch.inference_mode():
        y = fp4.mx_linear(x.clone(), w)
        assert y.is_inference() and torch.equal(y, want)
        b = fp4.MXTensor.quantize(w)
        assert torch.equal(b.matmul(x, out_dtype=torch.bfloat16), want)
    # weights quantised in inference mode, and inputs made there, go on outside it
    assert torch.equal(b.matmul(x, out_dtype=torch.bfloat16), want)
    (dw,) = torch.autograd.grad(fp4.mx_linear(y, w[:, :40]), w, torch.ones(24, 40, dtype=torch.bfloat16, device="cuda"))
    assert dw.shape == w.shape and not dw[:, 40:].any() and dw[:, :40].any()


@pytest.mark.parametrize("how", ["recomputed", "recomputed, reentrant", "saved on the host"])
def test_layer_under_checkpointing(how):
    """What the layer saves are the transposed operands: made again, or brought back from the host, they are the same."""
    from torch.utils.checkpoint import checkpoint
    x = dense(70, 160, torch.bfloat16, 252).cuda().requires_grad_()
    w = dense(96, 160, torch.float32, 253).cuda().requires_grad_()
    g = dense(70, 96, torch.bfloat16, 254).cuda()
    want = torch.autograd.grad(fp4.mx_linear(x, w), (x, w), g)
    for _ in range(2):
        x.grad = w.grad = None
        if how == "saved on the host":
            with torch.autograd.graph.save_on_cpu():
                y = fp4.mx_linear(x, w)
        else:
            y = checkpoint(fp4.mx_linear, x, w, use_reentrant="reentrant" in how)
        y.backward(g)
        assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])


def test_layer_as_a_graphed_callable():
    """Forward and backward captured by torch's own helper, replayed beside eager work."""
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.w = torch.nn.Parameter(dense(96, 512, torch.float32, 255))

        def forward(self, x):
            return fp4.mx_linear(x, self.w)

    layer = Layer().cuda()
    sample = dense(130, 512, torch.bfloat16, 256).cuda().requires_grad_()
    plain = Layer().cuda()
    graphed = torch.cuda.make_graphed_callables(layer, (sample,))
    for i in range(4):
        x = dense(130, 512, torch.bfloat16, 257 + i).cuda().requires_grad_()
        g = dense(130, 96, torch.bfloat16, 267 + i).cuda()
        y = graphed(x)
        got = torch.autograd.grad(y, (x, layer.w), g)
        torch.cuda.synchronize()
        ye = fp4.mx_linear(x, plain.w)
        want = torch.autograd.grad(ye, (x, plain.w), g)
        assert torch.equal(y, ye) and all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()
