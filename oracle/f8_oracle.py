"""fp64 CPU oracle for the e4m3 operators: the format, its quantiser, the norm, the products.

TEST INFRASTRUCTURE ONLY, like ``bgq_oracle``: the plain definitions in float64 with numpy, sharing no code with the
library. Codes and scales are the stored bytes.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 128


def code_values() -> np.ndarray:
    """What each of the 256 codes stands for: a sign, four bits of exponent (bias 7, 0: subnormal), three of fraction."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = -v if c & 128 else v
    return out


def values(q, scale, block_rows: int = 1) -> np.ndarray:
    """q uint8 [rows][cols], scale uint8 [rows/block_rows][cols/128] -> the values."""
    q, scale = np.asarray(q), np.asarray(scale)
    s = 2.0 ** (scale.astype(np.float64) - 127)
    s = np.repeat(np.repeat(s, block_rows, 0)[:q.shape[0]], BLOCK, 1)[:, :q.shape[1]]
    return code_values()[q] * s


def nearest_codes(x) -> np.ndarray:
    """The codes nearest to x (finite, at most 448 in size), halves to the even one, by search among all of them."""
    table = code_values()[:127]  # the codes of sizes rise with their value
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(table, a), 1, 126)
    below, above = a - table[hi - 1], table[hi] - a
    c = np.where(below < above, hi - 1, np.where(below > above, hi, np.where(hi % 2 == 0, hi, hi - 1)))
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def scale_byte(top: float) -> int:
    """The smallest power of two, from 2^-127 on, that leaves nothing of a block beyond 448."""
    e = -127
    while 448.0 * 2.0 ** e < top:
        e += 1
    return e + 127


def quantise(x, block_rows: int = 1):
    """x [rows][cols] float64 -> codes, scales."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    q = np.empty((rows, cols), dtype=np.uint8)
    s = np.empty((-(-rows // block_rows), -(-cols // BLOCK)), dtype=np.uint8)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            if np.isfinite(x[at]).all():
                s[i, j] = scale_byte(np.abs(x[at]).max())
                q[at] = nearest_codes(x[at] * 2.0 ** (127 - float(s[i, j])))
            else:
                s[i, j], q[at] = 127, 127
    return q, s


def norm(h, delta, rho, eps: float):
    """(h + delta, its RMSNorm times rho); rho None for ones."""
    h = np.asarray(h, dtype=np.float64) + (0.0 if delta is None else delta)
    a = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, a if rho is None else a * rho


def product(x, w):
    """x w^T, and what its rounding errors are counted in: the sum of the products' sizes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u
