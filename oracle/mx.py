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
