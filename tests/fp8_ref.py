"""8-bit floating point in blocks of 128 in numpy, 64-bit, straight from its
definition (test infrastructure only): every step is exact, so codes, scales and
values are compared bit for bit and products against fp64 sums."""
from __future__ import annotations

import numpy as np

# mantissa bits, exponent bias, largest value
FMT = {"f8e4m3": (3, 7, 448.0), "f8e5m2": (2, 15, 57344.0)}


def shapes(rows: int, K: int, block_rows: int = 1):
    return (rows, -(-K // 128) * 128), (-(-rows // block_rows), -(-K // 512) * 4)


def table(f8: str) -> np.ndarray:
    """The 256 values of the codes."""
    bits, bias, _ = FMT[f8]
    c = np.arange(128)
    e, m = c >> bits, (c & ((1 << bits) - 1)) / (1 << bits)
    v = np.where(e == 0, np.ldexp(m, 1 - bias), np.ldexp(1 + m, e - bias))
    if f8 == "f8e4m3":
        v[127] = np.nan
    else:
        v[124], v[125:] = np.inf, np.nan
    return np.concatenate([v, -v])


def scale_exponent(top: np.ndarray, f8: str) -> np.ndarray:
    """The smallest e with top <= largest * 2^e, in [-127, 127]; -127 for zero."""
    big = FMT[f8][2]
    m, ex = np.frexp(top)                              # top = m 2^ex, m in [1/2, 1); big = 0.875 * 2^b
    e = ex - np.frexp(big)[1] + (m > 0.875)
    return np.where(top > 0, np.clip(e, -127, 127), -127)


def quantize(x: np.ndarray, f8: str, block_rows: int = 1):
    """float64 [rows, K] -> (codes, scales); NaN comes out as 0x7f with its sign."""
    bits, bias, _ = FMT[f8]
    rows, K = x.shape
    kb, rb = -(-K // 128), -(-rows // block_rows)
    v = np.zeros((rb * block_rows, kb * 128))
    v[:rows, :K] = x
    v = v.reshape(rb, block_rows, kb, 128)
    finite = np.isfinite(v)
    top = np.abs(np.where(finite, v, 0.0)).max((1, 3))
    e = scale_exponent(top, f8)
    t = np.ldexp(np.abs(np.where(finite, v, 0.0)), -e[:, None, :, None])
    # the spacing of the values around t, and t in units of it, halves to even
    _, ex = np.frexp(t)
    step = np.maximum(ex - 1, 1 - bias) - bits
    n = np.rint(np.ldexp(t, -step)).astype(np.int64)   # below 2^(bits + 1), or equal to it: the next binade
    up = n >= (2 << bits)
    step, n = step + up, np.where(up, n >> 1, n)
    field = np.where(n >= (1 << bits), step + bits + bias, 0)
    code = (field << bits) + np.where(n >= (1 << bits), n - (1 << bits), n)
    code = np.where(np.isnan(v), 127, np.where(np.isinf(v), 124 if f8 == "f8e5m2" else 127, code))
    code = (code | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8).reshape(rb * block_rows, kb * 128)[:rows]
    scales = np.zeros((rb, -(-K // 512) * 4), np.uint8)
    scales[:, :kb] = e + 127
    return np.ascontiguousarray(code), scales


def values(codes: np.ndarray, scales: np.ndarray, K: int, f8: str, block_rows: int = 1) -> np.ndarray:
    """float64 [rows, K] of codes and scales."""
    rows = codes.shape[0]
    kb = codes.shape[1] // 128
    s = np.ldexp(1.0, scales[:, :kb].astype(np.int64) - 127)
    s = np.where(scales[:, :kb] == 255, np.nan, s)
    s = np.repeat(np.repeat(s, 128, 1), block_rows, 0)[:rows]
    return (table(f8)[codes] * s)[:, :K]


def random_packed(rng, rows: int, K: int, f8: str, block_rows: int = 1, lo: int = 118, hi: int = 128):
    """Random finite codes (padding zero) and scale bytes in [lo, hi] (padding 0 or 255)."""
    (_, kp), (rb, kw) = shapes(rows, K, block_rows)
    ok = np.flatnonzero(np.isfinite(table(f8))).astype(np.uint8)
    codes = rng.choice(ok, (rows, kp)).astype(np.uint8)
    codes[:, K:] = 0
    scales = rng.integers(lo, hi + 1, (rb, kw), dtype=np.uint8)
    scales[:, kp // 128:] = rng.choice(np.array([0, 255], np.uint8), (rb, kw - kp // 128))
    return codes, scales
