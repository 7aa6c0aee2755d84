"""MXFP4 products with an epilogue and of experts: what the calls do to the memory, streams and gradients around them."""
import numpy as np
import pytest
import torch

from tests import mx_reference as ref
from tests.mx_reference import dense, f64

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu

M, N, K, E = 70, 96, 128, 3


def leaves(*key, types=(torch.bfloat16, torch.float32, torch.float32, torch.bfloat16)):
    """x, w, bias, residual of a layer of E experts."""
    x, w = dense(M, K, types[0], 1, *key), dense(E * N, K, types[1], 2, *key, scale=0.2).reshape(E, N, K)
    return [t.requires_grad_() for t in (x, w, dense(E, N, types[2], 3, *key), dense(M, N, types[3], 4, *key))]


OFF = [0, 30, 30, 64]


def grouped(x, w, b, r, name="silu"):
    return fp4.mx_grouped_linear(x, w, torch.tensor(OFF, device="cuda"), bias=b, activation=name, residual=r)


def one(x, w, b, r, name="silu"):
    return fp4.mx_linear(x, w[0], bias=b[0], activation=name, residual=r)


@pytest.mark.parametrize("call", [grouped, one])
@pytest.mark.parametrize("how", ["host", "reentrant", "not reentrant"])
def test_layers_under_checkpointing(call, how):
    from torch.utils.checkpoint import checkpoint
    t, g = leaves(), dense(M, N, torch.bfloat16, 5)
    want = torch.autograd.grad(call(*t), t, g)
    again = [v.detach().clone().requires_grad_() for v in t]
    if how == "host":
        with torch.autograd.graph.save_on_cpu():
            y = call(*again)
    else:
        y = checkpoint(call, *again, use_reentrant=how == "reentrant")
    y.backward(g)
    for p, q in zip(again, want):
        assert torch.equal(p.grad, q)


@pytest.mark.parametrize("call", [grouped, one])
def test_layers_without_gradients(call):
    t = leaves(6)
    want = call(*t).detach()
    with torch.inference_mode():
        y = call(*t)
        assert y.is_inference() and torch.equal(y, want)
        held = [v.clone() for v in t]
    assert torch.equal(call(*held), want) and not call(*held).requires_grad
    with torch.no_grad():
        assert torch.equal(call(*t), want)


def test_layer_of_experts_as_a_graphed_callable():
    t = leaves(7)

    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.w, self.b = torch.nn.Parameter(t[1].detach().clone()), torch.nn.Parameter(t[2].detach().clone())
            self.register_buffer("off", torch.tensor(OFF, device="cuda"))

        def forward(self, x):
            return fp4.mx_grouped_linear(x, self.w, self.off, bias=self.b, activation="gelu")
    layer, eager = Layer(), Layer()
    graphed = torch.cuda.make_graphed_callables(layer, (t[0].detach().clone().requires_grad_(),))
    for i in range(4):
        x = dense(M, K, torch.bfloat16, 8, i).requires_grad_()
        x2, g = x.detach().clone().requires_grad_(), dense(M, N, torch.bfloat16, 9, i)
        y, y2 = graphed(x), eager(x2)
        got = torch.autograd.grad(y, (x, *graphed.parameters()), g)
        want = torch.autograd.grad(y2, (x2, *eager.parameters()), g)
        assert torch.equal(y, y2)
        for p, q in zip(got, want):
            assert torch.equal(p, q)
        torch.cuda.synchronize()


def test_types_of_every_input_and_gradient():
    f32, bf16, f16 = torch.float32, torch.bfloat16, torch.float16
    g = dense(M, N, f32, 10)
    for i, types in enumerate(((bf16, f16, f32, f32), (f16, bf16, bf16, f32), (f32, f16, bf16, f16), (bf16, f32, f16, f16))):
        t = leaves(11, i, types=types)
        for call in (grouped, one):
            y = call(*t, name="gelu")
            assert y.dtype == types[0]
            grads = torch.autograd.grad(y, t, g.to(types[0]))
            assert [v.dtype for v in grads] == list(types) and torch.equal(grads[3], g.to(types[0]).to(types[3]))
            # the bias's and the residual's type have no say in the others: the values of both are the same
            u = [t[0], t[1], t[2].detach().float().requires_grad_(), t[3].detach().float().requires_grad_()]
            z = call(*u, name="gelu")
            assert torch.equal(z, y)
            other = torch.autograd.grad(z, u, g.to(types[0]))
            assert torch.equal(other[0], grads[0]) and torch.equal(other[1], grads[1]) and torch.equal(other[2].to(types[2]), grads[2])


def test_inputs_of_every_layout():
    t, g = leaves(12), dense(M, N, torch.bfloat16, 13)
    want = [grouped(*t), *torch.autograd.grad(grouped(*t), t, g)]
    far = [dense(K, M, torch.bfloat16, 14).T, dense(N * K, E, torch.float32, 15).reshape(N, K, E).permute(2, 0, 1), dense(N, 2 * E, torch.float32, 16).T[::2],
           dense(N, M, torch.bfloat16, 17).T]
    with torch.no_grad():
        for f, v in zip(far, t):
            assert f.shape == v.shape and not f.is_contiguous()
            f.copy_(v)
    far = [f.requires_grad_() for f in far]
    for p, q in zip([grouped(*far), *torch.autograd.grad(grouped(*far), far, g.T.contiguous().T)], want):
        assert torch.equal(p, q)
    with torch.no_grad():
        neg = [torch._neg_view((-v).contiguous()) for v in t]
        assert all(v.is_neg() for v in neg) and torch.equal(grouped(*neg), want[0]) and torch.equal(one(*neg), one(*t))
        # one row without an axis for it, and more axes
        x, r = t[0][3], t[3][3]
        y = fp4.mx_grouped_linear(x, t[1], torch.tensor([0, 1, 1, 1], device="cuda"), bias=t[2], activation="silu", residual=r)
        assert y.shape == (N,) and torch.equal(y, want[0][3])
        y = fp4.mx_grouped_linear(t[0].reshape(2, 5, 7, K), t[1], torch.tensor(OFF, device="cuda"), bias=t[2], activation="silu",
                                  residual=t[3].reshape(2, 5, 7, N))
        assert torch.equal(y.reshape(M, N), want[0])


def test_written_tensors_count_as_changed():
    x, w, b, r = (v.detach() for v in leaves(18))
    off = torch.tensor(OFF, device="cuda")
    q, d = fp4.MXTensor.quantize(w), fp4.MXTensor.quantize(w[0])
    a, scale = fp4.MXTensor.quantize(x), torch.ones(N, device="cuda", requires_grad=True)
    for write in (lambda y: q.grouped_matmul(x, off, out=y), lambda y: q.grouped_matmul(a, off, out=y), lambda y: d.matmul(a, out=y, bias=b[0]),
                  lambda y: d.matmul(x, out=y, residual=y),
                  lambda y: fp4.w4a4_grouped_linear(M, N, K, x, q.codes, q.scales, off, y),
                  lambda y: fp4.w4a4_grouped_matmul(M, N, K, a.codes, a.scales, q.codes, q.scales, off, y)):
        y = torch.randn(M, N, device="cuda")
        loss = (y * scale).sum()
        write(y)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    q.grouped_matmul(x, off, bias=b, residual=r, activation="relu")
    d.matmul(x, bias=b[0], residual=r)
    assert all(t._version == 0 for t in (off, q.codes, q.scales, a.codes)) and r._version == dense(M, N, torch.bfloat16, 4, 18)._version


def test_a_stream_of_another_gpu_is_refused():
    x, w, b, r = (v.detach() for v in leaves(19))
    off, q = torch.tensor(OFF, device="cuda"), fp4.MXTensor.quantize(w)
    side = torch.cuda.Stream()

    class Elsewhere:                                           # as a torch stream of a second GPU looks
        cuda_stream, device = side.cuda_stream, torch.device("cuda", x.device.index + 1)
    y = torch.empty(M, N, device="cuda")
    a = fp4.MXTensor.quantize(x)
    for call in (lambda s: q.grouped_matmul(x, off, stream=s), lambda s: q.grouped_matmul(a, off, residual=r, stream=s),
                 lambda s: fp4.w4a4_grouped_linear(M, N, K, x, q.codes, q.scales, off, y, stream=s),
                 lambda s: fp4.w4a4_grouped_matmul(M, N, K, a.codes, a.scales, q.codes, q.scales, off, y, stream=s)):
        with pytest.raises(ValueError, match="stream belongs"):
            call(Elsewhere())


def test_a_graph_keeps_a_given_workspace_of_its_own():
    """Two graphs captured with a workspace each, replayed by turns on two streams."""
    m, n, k = 40, 200, 8192
    w = fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 20))
    b = dense(1, n, torch.float32, 21)[0]
    graphs = []
    for i in range(2):
        x = dense(m, k, torch.bfloat16, 22, i)
        ws = torch.empty(fp4.w4a4_linear_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda").fill_(255)
        want = w.matmul(x, bias=b, activation="gelu")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = w.matmul(x, workspace=ws, bias=b, activation="gelu")
        graphs.append((graph, x, ws, y, want, side))
    for _ in range(4):
        for graph, _, _, y, _, side in graphs:
            with torch.cuda.stream(side):
                y.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, _, _, y, want, _ in graphs:
            assert torch.equal(y, want)


def test_the_same_rows_twice():
    """A token sent to one expert twice, and one expert's weights standing for two."""
    x, w, b, r = (v.detach() for v in leaves(23))
    off = torch.tensor([0, 40, 40, 70], device="cuda")
    rows = torch.tensor([5] * 3 + list(range(37)) + [5] * 30, device="cuda")
    q = fp4.MXTensor.quantize(torch.stack([w[1], w[0], w[1]]))
    y = q.grouped_matmul(x[rows], off, bias=b[[1, 0, 1]], activation="gelu")
    z, ez = ref.with_bias(*ref.product(ref.values(x[rows]), ref.values(w[1]), K), f64(b[1]))
    ref.check(y, *ref.out(z, ez, "gelu", None, torch.float32))
    assert torch.equal(y[0], y[40]) and np.unique(f64(y)[[0, 1, 2, 8, *range(40, 70)]], axis=0).shape[0] == 1


def test_a_residual_that_overlaps_the_output_is_refused():
    """The same memory at the same place is added to; any other overlap would have one tile read what another wrote."""
    x, w, b, _ = (v.detach() for v in leaves(24))
    d, q, off = fp4.MXTensor.quantize(w[0]), fp4.MXTensor.quantize(w), torch.tensor(OFF, device="cuda")
    bad, good = [], []
    flat = torch.zeros((M + 2) * N + 8, device="cuda")
    at = lambda start: flat[start:start + M * N].view(M, N)  # noqa: E731
    bad += [(at(N), at(0)), (at(0), at(N)), (at(0), at(1)), (at(3), at(0)), (at(0), at(2 * N))]
    wide = torch.zeros(M + 1, 3 * N, device="cuda")
    col = lambda start, row=0: wide[row:row + M, start:start + N]  # noqa: E731
    bad += [(col(0), col(N - 1)), (col(N), col(1)), (col(5), col(5, 1)), (col(2 * N, 0), col(2 * N - 3, 1)), (col(5, 1), col(9))]
    good += [(col(0), col(N)), (col(2 * N), col(N)), (col(0, 1), col(2 * N)), (col(2 * N), col(0, 1)), (col(7), col(7))]
    half = torch.zeros(4 * M * N, dtype=torch.bfloat16, device="cuda")
    bad += [(half[:2 * M * N].view(torch.float32).view(M, N), half[M * N:2 * M * N].view(M, N))]
    good += [(half[:2 * M * N].view(torch.float32).view(M, N), half[2 * M * N:3 * M * N].view(M, N)), (at(0), at(0))]
    for y, r in bad:
        for call in (lambda: d.matmul(x, out=y, residual=r), lambda: q.grouped_matmul(x, off, out=y, residual=r),  # noqa: B023
                     lambda: fp4.w4a4_linear(M, N, K, x, d.codes, d.scales, y, residual=r)):  # noqa: B023
            with pytest.raises(ValueError, match="share"):
                call()
    for y, r in good:
        want = d.matmul(x, out_dtype=y.dtype, bias=b[0], residual=r.clone())
        assert torch.equal(d.matmul(x, out=y, bias=b[0], residual=r), want)
        y.zero_()
