"""MXFP4 in NumPy, from the format's definition (OCP Microscaling Formats
v1.0: E2M1 elements in blocks of 32, one E8M0 scale per block).

Independent of the CUDA library: elements are rounded by searching the grid.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_e2m1(y: np.ndarray) -> np.ndarray:
    """Codes of the grid values nearest to y (float64), ties to the even code,
    clamped at 6; the sign of -0.0 is kept."""
    a = np.minimum(np.abs(y), 6.0)
    hi = np.clip(np.searchsorted(GRID, a, side="left"), 0, 7)
    lo = np.maximum(hi - 1, 0)
    to_lo, to_hi = a - GRID[lo], GRID[hi] - a
    even = np.where(lo % 2 == 0, lo, hi)
    code = np.where(to_lo < to_hi, lo, np.where(to_hi < to_lo, hi, even))
    return (code | (np.signbit(y).astype(np.int64) << 3)).astype(np.uint8)


def quantize(x: np.ndarray):
    """x [rows, cols] -> (codes [rows, ceil32(cols)/2], scale bytes
    [rows, ceil(cols/32)])."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = np.zeros((rows, nb * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, nb, BLOCK)
    amax = np.abs(v).max(axis=2)
    bad = ~np.isfinite(v).all(axis=2)
    _, e = np.frexp(np.where(bad | (amax == 0), 1.0, amax))       # amax = m 2^e, m in [1/2, 1)
    exp = np.maximum(np.where(amax == 0, -127, e - 1 - 2), -127)
    y = np.ldexp(np.where(bad[:, :, None], 0.0, v), -exp[:, :, None])
    code = np.where(bad[:, :, None], 0, round_e2m1(y)).reshape(rows, -1).astype(np.uint8)
    scale = np.where(bad, 255, exp + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def dequantize(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """float64 values [rows, cols]."""
    rows = codes.shape[0]
    c = np.stack([codes & 15, codes >> 4], axis=2).reshape(rows, -1)
    v = np.where(c & 8, -GRID[c & 7], GRID[c & 7])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * np.repeat(s, BLOCK, axis=1))[:, :cols]


def tiled_index(rows: int, cols: int) -> np.ndarray:
    """idx[r, b] = byte of (row r, block b) in the tiled scale layout."""
    nb = -(-cols // BLOCK)
    r, b = np.arange(rows)[:, None], np.arange(nb)[None, :]
    return ((r // 128) * (-(-nb // 4)) + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4


def to_tiled(scales: np.ndarray, cols: int) -> np.ndarray:
    rows, nb = scales.shape
    out = np.zeros(-(-rows // 128) * (-(-nb // 4)) * 512, np.uint8)
    out[tiled_index(rows, cols)] = scales
    return out
