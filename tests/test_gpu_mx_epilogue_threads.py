"""Threads that call MXFP4 products with an epilogue, products of experts and both layers at once, each on a stream of its own: every
call is counted, every error raised."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from tests.mx_reference import dense

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")
pytestmark = pytest.mark.gpu
ROUNDS = 15


def product(m, n, k):
    w, x = fp4.MXTensor.quantize(dense(n, k, torch.bfloat16, 1)), dense(m, k, torch.bfloat16, 2)
    kw = dict(bias=dense(1, n, torch.float32, 3)[0], activation="gelu", residual=dense(n, m, torch.bfloat16, 4).T)
    return lambda: (w.matmul(x, **kw),)


def experts(t, n, k, e):
    w, x = fp4.MXTensor.quantize(dense(e * n, k, torch.bfloat16, 5)), dense(k, t, torch.bfloat16, 6).T
    off = torch.linspace(0, t - 2, e + 1, device="cuda").int()
    bias = dense(e, n, torch.float32, 7)
    return lambda: (w.grouped_matmul(x, off, bias=bias, activation="silu"),)


def layer(m, n, k):
    x, w = dense(m, k, torch.bfloat16, 8).requires_grad_(), dense(n, k, torch.float32, 9).requires_grad_()
    b, g = dense(1, n, torch.float32, 10)[0].requires_grad_(), dense(m, n, torch.bfloat16, 11)

    def step():
        y = fp4.mx_linear(x, w, bias=b, activation="silu")
        return y.detach(), *torch.autograd.grad(y, (x, w, b), g)
    return step


def layer_of_experts(t, n, k, e):
    x, w = dense(t, k, torch.bfloat16, 12).requires_grad_(), dense(e * n, k, torch.float32, 13).reshape(e, n, k).requires_grad_()
    b, g = dense(e, n, torch.float32, 14).requires_grad_(), dense(t, n, torch.bfloat16, 15)
    off = torch.linspace(1, t, e + 1, device="cuda").long()

    def step():
        y = fp4.mx_grouped_linear(x, w, off, bias=b, activation="gelu_tanh")
        return y.detach(), *torch.autograd.grad(y, (x, w, b), g)
    return step


@pytest.mark.parametrize("calls", [lambda: [product(40, 200, 8192)] * 2, lambda: [experts(300, 200, 512, 8)] * 2,
                                   lambda: [product(9, 512, 1024), experts(12, 96, 256, 4), product(300, 520, 512), experts(700, 300, 256, 6)],
                                   lambda: [layer(150, 96, 256)] * 2 + [layer_of_experts(200, 96, 128, 5)] * 2],
                         ids=["product", "experts", "both", "layers"])
def test_at_once(calls):
    calls = calls()
    want = [call() for call in calls]
    torch.cuda.synchronize()

    def run(i):
        done, own = 0, torch.cuda.Stream()
        with torch.cuda.stream(own):
            for _ in range(ROUNDS):
                got = calls[i]()
                own.synchronize()
                assert len(got) == len(want[i])
                for p, q in zip(got, want[i]):
                    assert torch.equal(p, q)
                done += 1
        own.synchronize()
        return done

    with ThreadPoolExecutor(len(calls)) as pool:
        assert [f.result(timeout=60) for f in [pool.submit(run, i) for i in range(len(calls))]] == [ROUNDS] * len(calls)
