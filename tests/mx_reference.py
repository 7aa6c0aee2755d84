"""FP64 references on the GPU's own tensors for the GPU tests of products with an epilogue and of experts' products: values by the
oracle, sums by plain matrix products in 64 bits, tolerances by arithmetic."""
import numpy as np
import torch

from oracle import mx

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}        # half the smallest step
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().cpu().double().numpy()


def dense(m, k, dtype, *key, scale=1.0):
    """Normal values with rows of different size and some zeros."""
    r = np.random.default_rng([20261208, m, k, *key])
    x = r.standard_normal((m, k)) * np.exp2(r.integers(-3, 4, (m, 1))) * scale
    x[r.random((m, k)) < 0.02] = 0.0
    return torch.from_numpy(x).to(dtype).cuda()


def values(x):
    """The values of the MXFP4 form of x, blocks along the last axis."""
    return mx.dequant(*mx.quantize(f64(x)), x.shape[-1])


def mm(a, b):
    """a b^T of FP64 arrays, on the GPU."""
    return torch.mm(torch.from_numpy(np.ascontiguousarray(a)).cuda(), torch.from_numpy(np.ascontiguousarray(b)).cuda().T).cpu().numpy()


def product(a, b, k):
    """(A B^T, how far its FP32 evaluation may be off)."""
    return mm(a, b), mx.sum_bound(k, mm(np.abs(a), np.abs(b)))


def with_bias(z, ez, bias):
    """The sum with a bias added: one more rounding."""
    if bias is None:
        return z, ez
    z = z + bias
    return z, ez + 2.0 ** -24 * (np.abs(z) + ez)


def out(z, ez, name, residual, dtype):
    """(y, tolerance): every f rises by at most 1.13 times what z does; the residual's addition and the output round once each."""
    f, ef = mx.activation(name, z)
    y, tol = f, 1.13 * ez + ef
    if residual is not None:
        y = f + residual
        tol = tol + 2.0 ** -24 * (np.abs(y) + tol)
    return y, tol + HALF[dtype] * (np.abs(y) + tol) + TINY[dtype]


def check(got, want, tol, label=""):
    got = f64(got)
    assert got.shape == want.shape, label
    ok = np.abs(got - want) <= tol
    assert ok.all(), f"{label}: {np.count_nonzero(~ok)} off, worst {np.max(np.abs(got - want) / np.maximum(tol, 1e-300))} of the tolerance"


def round_to(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


def gradient_interval(g, z, ez, name, dtype):
    """(low, high) of D = g f'(z) in its type, z being known to ez: f' of each activation changes by at most 1.2 of what z does
    (relu's by all of it where 0 lies in reach), and rounding to a type is monotone."""
    s, es = mx.slope(name, z)
    if name == "relu":
        lo, hi = (z - ez > 0) * 1.0, (z + ez > 0) * 1.0
    else:
        e = es + (0 if name is None else 1.2 * ez)
        lo, hi = s - e, s + e
    a, b = g * lo, g * hi
    lo, hi = np.minimum(a, b), np.maximum(a, b)
    if name not in (None, "relu"):  # the product's own rounding in FP32
        lo, hi = lo - 2.0 ** -24 * np.abs(lo), hi + 2.0 ** -24 * np.abs(hi)
    return round_to(lo, dtype), round_to(hi, dtype)


def interval_product(low, high, b, k):
    """(middle, tolerance) of Q(D) B^T in FP32, D in [low, high] elementwise, blocks along its rows, B's values exact."""
    lo, hi = mx.quantize_interval(low, high)
    mid, rad = (lo + hi) / 2, (hi - lo) / 2
    return mm(mid, b), mm(rad, np.abs(b)) + mx.sum_bound(k, mm(np.maximum(np.abs(lo), np.abs(hi)), np.abs(b)))


def rounded(want, tol, dtype):
    return tol + HALF[dtype] * (np.abs(want) + tol) + TINY[dtype]


def bias_gradient(g, z, ez, name, dtype):
    """(sum of g f'(z) over the rows, tolerance): each value as above without rounding to g's type; 32 rows are summed one
    after the other, up to 8 of their sums likewise, in FP32, the rest in FP64, and the result is rounded once."""
    s, es = mx.slope(name, z)
    e = np.abs(g) * (es + (0 if name is None else 1.2 * ez) + 2.0 ** -24 * np.abs(s))
    if name == "relu":
        e = np.abs(g) * (np.abs(z) <= ez)
    d = g * s
    want = d.sum(axis=0)
    tol = e.sum(axis=0) + 41 * 2.0 ** -24 * (np.abs(d) + e).sum(axis=0)
    return want, rounded(want, tol + 2.0 ** -24 * (np.abs(want) + tol), dtype)
