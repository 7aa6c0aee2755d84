"""MXFP4 (OCP Microscaling Formats specification 1.0, E2M1 elements and one E8M0 scale per 32 values) in FP64 numpy:
quantisation along the last axis, its inverse, and products. Test infrastructure; shares nothing with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 32
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(k: int) -> int:
    return -(-k // BLOCK)


def quantize(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """x [R, K] -> codes uint8 [R, 16 ceil(K/32)], scales uint8 [R, ceil(K/32)], blocks along K padded with zeros."""
    r, k = x.shape
    nb = blocks(k)
    v = np.zeros((r, nb * BLOCK))
    v[:, :k] = x
    v = v.reshape(r, nb, BLOCK)
    finite = np.isfinite(v).all(axis=2)
    v = np.where(finite[..., None], v, 0.0)
    amax = np.abs(v).max(axis=2)
    _, e = np.frexp(amax)                                  # amax = f 2^e, f in [1/2, 1): floor(log2) = e - 1
    s = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    q = np.abs(v) / np.ldexp(1.0, s - 127)[..., None]
    away = np.abs(q[..., None] - LEVELS)
    best = away.min(axis=-1)
    near = away == best[..., None]                         # one level, or two neighbours of which one code is even
    even = np.arange(8) % 2 == 0
    code = np.where((near & even).any(axis=-1) & (near.sum(axis=-1) == 2), (near & even).argmax(axis=-1), near.argmax(axis=-1))
    code = code + 8 * np.signbit(v)
    code = np.where(finite[..., None], code, 0).reshape(r, nb * BLOCK).astype(np.uint8)
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8), np.where(finite, s, 255).astype(np.uint8)


def dequant(codes: np.ndarray, scales: np.ndarray, k: int | None = None) -> np.ndarray:
    """FP64 values of codes and scales (the first k of each row)."""
    c = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = LEVELS[c & 7] * np.where(c >= 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * np.repeat(s, BLOCK, axis=1))[:, :k]


def product(a: np.ndarray, b: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(A B^T, |A| |B|^T) in FP64."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def sum_bound(k: int, magnitude: np.ndarray) -> np.ndarray:
    """How far an FP32 evaluation of a depth-k product may be from the exact one, `magnitude` = |A| |B|^T.

    The products of E2M1 levels and powers of two are exact. The sum takes one matrix instruction per 128 positions;
    each adds its 128 products and the running sum, aligned to the largest of them and cut at FP32's 24 bits, once per
    group of 32: at most four cuts of 2^-23 of a partial sum of magnitudes. Joining up to 16 partial sums of waves or K
    parts, one rounding of 2^-24 each, comes on top."""
    steps = -(-k // 128)
    return (4 * steps + 16) * 2.0 ** -23 * magnitude


# --------------------------------------------------------------------------------- what follows a product

ACTIVATIONS = (None, "relu", "silu", "gelu", "gelu_tanh")
STEP = 2.0 ** -23


def _logistic(v: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def activation(name: str | None, z: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """f(z) in FP64 and how far an FP32 evaluation at the FP32 number z may be from it.

    silu and gelu by tanh are z s(v), v = z or 2 sqrt(2 / pi) (z + 0.044715 z^3), s the logistic function: v is good to four
    roundings, which 2^u turns into a relative error of |v| times theirs, the logistic function takes up by a factor 1 - s, and
    2^u, the sum, the reciprocal and the product add at most four steps. gelu is max(z, 0) less |z| times the normal
    distribution's tail t: exp(-z^2 / 2) is good to z^2 / 2 times three roundings, the polynomial of degree 7 in a number of
    (0, 1] with coefficients of both signs (their magnitudes sum to at most four times its value) to 32 steps, its fit (1.25e-7
    where a step is 1.19e-7) to two, 2^u to one, and the tail's two products to half a step each: 36 in all."""
    if name is None:
        return z, np.zeros_like(z)
    if name == "relu":
        return np.maximum(z, 0), np.zeros_like(z)
    if name == "gelu":
        from scipy.special import ndtr
        tail = np.abs(z) * ndtr(-np.abs(z))
        f = np.maximum(z, 0) - tail
        return f, STEP * (tail * (36 + z * z) + np.abs(f)) + 2.0 ** -120
    v = z if name == "silu" else 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    s = _logistic(v)
    return z * s, STEP * np.abs(z * s) * (2 * np.abs(v) * _logistic(-v) + 4) + 2.0 ** -120


def slope(name: str | None, z: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """f'(z) and how far an FP32 evaluation may be from it: activation()'s bounds for s and the tail; the product z s (1 - s) q
    takes s, its complement and four more roundings."""
    one = np.ones_like(z)
    if name is None:
        return one, 0 * one
    if name == "relu":
        return (z > 0) * one, 0 * one
    if name == "gelu":
        from scipy.special import ndtr
        tail, density = ndtr(-np.abs(z)), z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        return ndtr(z) + density, STEP * (tail * (36 + z * z) + np.abs(density) * (8 + z * z) + (z > 0)) + 2.0 ** -120
    c = 1.0 if name == "silu" else 2 * np.sqrt(2 / np.pi)
    k = 0.0 if name == "silu" else 0.044715
    v, q = c * (z + k * z ** 3), c * (1 + 3 * k * z * z)
    s, t = _logistic(v), _logistic(-v)
    d = z * s * t * q
    return s + d, STEP * (s * (2 * np.abs(v) * t + 4) + np.abs(d) * (2 * np.abs(v) + 12)) + 2.0 ** -110


def quantize_interval(low: np.ndarray, high: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """The least and the largest values that the MXFP4 form of x may stand for, blocks along the last axis, where each element
    of x is only known to lie in [low, high]: rounding is monotone at a given scale, and a block whose largest magnitude may
    lie on either side of a power of two has the values at both scales. Where it may lie further apart, any scale between may be the
    block's: rounding to the nearest level at most doubles a magnitude (0.25 to 0.5), whatever the scale."""
    r, k = low.shape
    least = np.where((low <= 0) & (high >= 0), 0.0, np.minimum(np.abs(low), np.abs(high)))
    most = np.maximum(np.abs(low), np.abs(high))
    shape = (r, blocks(k), BLOCK)

    def wide(x):
        v = np.zeros((r, blocks(k) * BLOCK))
        v[:, :k] = x
        return v.reshape(shape)

    def scale(a):
        amax = wide(a).max(axis=2)
        _, e = np.frexp(amax)
        return np.where(amax > 0, np.maximum(e - 1 - 2, -127), -127)

    far = np.repeat(scale(most) - scale(least) > 1, BLOCK, axis=1)[:, :k]
    lowest, highest = np.where(far, np.minimum(2 * low, 0), np.inf), np.where(far, np.maximum(2 * high, 0), -np.inf)
    bounds = []
    for s in (scale(least), scale(most)):
        p = np.ldexp(1.0, s)[..., None]
        for x in (low, high):
            q = np.abs(wide(x)) / p
            # halves go to the even code: 0, 1, 2 and 4 take theirs from below and above
            level = (0.5 * (q > 0.25) + 0.5 * (q >= 0.75) + 0.5 * (q > 1.25) + 0.5 * (q >= 1.75) + 1.0 * (q > 2.5) + 1.0 * (q >= 3.5)
                     + 2.0 * (q > 5.0))
            bounds.append((np.sign(wide(x)) * level * p).reshape(r, -1)[:, :k])
    return np.minimum(np.minimum.reduce(bounds), lowest), np.maximum(np.maximum.reduce(bounds), highest)
