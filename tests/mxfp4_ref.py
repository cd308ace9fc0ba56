"""The MXFP4 format in numpy, 64-bit, straight from its definition (test
infrastructure only): every step is exact, so codes and values are compared
bit for bit and products against fp64 sums."""
from __future__ import annotations

import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def groups(K: int) -> int:
    return -(-K // 128)


def quantize(x: np.ndarray):
    """float64 [rows, K] -> (codes [rows, 64 G], scales [rows, 4 G])."""
    rows, K = x.shape
    G = groups(K)
    v = np.zeros((rows, G * 128))
    v[:, :K] = x
    v = v.reshape(rows, G * 4, 32)
    finite = np.isfinite(v).all(-1)
    top = np.where(finite, np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1), 0.0)
    _, ex = np.frexp(top)                              # top in [2^(ex-1), 2^ex)
    e = np.where(top > 0, np.clip(ex - 3, -127, 127), -127)
    t = np.ldexp(np.abs(np.where(finite[..., None], v, 0.0)), -e[..., None])
    d = np.abs(t[..., None] - MAGS)
    best = d.min(-1, keepdims=True)
    # the nearest magnitude; of two equally near ones the even code
    cand = np.where(d == best, np.where(np.arange(8) % 2 == 0, 0, 1), 2)
    code = cand.argmin(-1).astype(np.uint8)
    code |= (np.signbit(v).astype(np.uint8) << 3)
    code[~finite] = 0
    code = code.reshape(rows, -1)
    scale = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def values(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """float64 [rows, K] of packed codes and scales."""
    rows = codes.shape[0]
    nib = np.empty((rows, codes.shape[1] * 2), np.uint8)
    nib[:, 0::2] = codes & 15
    nib[:, 1::2] = codes >> 4
    v = np.where(nib & 8, -1.0, 1.0) * MAGS[nib & 7]
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s = np.where(scales == 255, np.nan, s)
    return (v * np.repeat(s, 32, axis=1))[:, :K]


def random_packed(rng, rows: int, K: int, lo: int = 118, hi: int = 128):
    """Random codes (padding zero) and scale bytes in [lo, hi]."""
    G = groups(K)
    nib = rng.integers(0, 16, (rows, G * 128), dtype=np.uint8)
    nib[:, K:] = 0
    codes = nib[:, 0::2] | (nib[:, 1::2] << 4)
    scales = rng.integers(lo, hi + 1, (rows, G * 4), dtype=np.uint8)
    scales[:, -(-K // 32):] = 0
    return codes, scales
