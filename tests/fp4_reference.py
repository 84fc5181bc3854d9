"""The microscaled 4-bit rule and product in 64 bits, on numpy arrays: by
distance to the grid, apart from any bit trick of the kernels."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quant(x: np.ndarray):
    """float64 x [M, K] -> (codes uint8 [M, K/2], scale bytes uint8 [M, K/32])."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32).astype(np.float64)
    bad = ~np.isfinite(b).all(-1)
    a = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    mant, exp = np.frexp(a)                              # a = mant * 2^exp, mant in [1/2, 1)
    e = np.where(a > 0, np.clip(exp - 1 - 2, -127, 127), -127)
    v = np.where(bad[..., None], 0.0, b) / (2.0 ** e)[..., None]
    # nearest grid value; of two equally near the one with the even code
    d = np.abs(np.abs(v)[..., None] - GRID)
    d = np.where(np.arange(8) % 2 == 1, np.nextafter(d, np.inf), d)
    code = d.argmin(-1).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(M, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def dequant(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values in float64 [M, K]; NaN in blocks of scale byte 255."""
    M = codes.shape[0]
    n = np.stack((codes & 15, codes >> 4), -1).reshape(M, -1, 32)
    v = np.where(n & 8, -1.0, 1.0) * GRID[n & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(M, -1)


def product(x: np.ndarray, w: np.ndarray):
    """(x @ w^T, |x| @ |w|^T) of dequantized float64 operands; NaN where a NaN
    block takes part."""
    nan = np.isnan(x).any(1)[:, None] | np.isnan(w).any(1)[None, :]
    x, w = np.nan_to_num(x), np.nan_to_num(w)
    return np.where(nan, np.nan, x @ w.T), np.abs(x) @ np.abs(w).T
