"""FP8: E4M3 codes with one fp32 scale for each block of 128, products and products grouped by expert.

Test infrastructure only (see the package docstring).  A block is 128 consecutive k of a row (block_rows 1) or 128
rows by 128 k (block_rows 128); the last one along either may be shorter.
"""
from __future__ import annotations

import math

import numpy as np

from .fp4 import e4m3_value

BLOCK = 128
_MAGS = np.array([float(e4m3_value(c)) for c in range(127)])   # 0 .. 448, ascending, code = index
_MIDS = (_MAGS[1:] + _MAGS[:-1]) / 2


def encode(y) -> np.ndarray:
    """E4M3 codes nearest to y (fp64, |y| below the middle between 448 and the 480 that is not there), ties to the
    even code, the sign bit that of y."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    lo = np.searchsorted(_MIDS, a, side="left")     # the middles below a
    hi = np.searchsorted(_MIDS, a, side="right")    # and those not above it: one more at a tie
    code = np.where(lo == hi, lo, lo + (lo & 1))
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def encode_scalar(y: float) -> int:
    """The same by the distance to every magnitude."""
    best = min(range(127), key=lambda i: (abs(_MAGS[i] - abs(y)), i & 1))
    return best | (128 if math.copysign(1.0, y) < 0 else 0)


def decode(codes) -> np.ndarray:
    """fp64 values of E4M3 bytes."""
    c = np.asarray(codes).astype(np.int64)
    return np.where(c & 127 == 127, np.nan, np.append(_MAGS, 0.0)[c & 127] * np.where(c >= 128, -1.0, 1.0))


def scale_shape(shape, block_rows):
    return (*shape[:-2], -(-shape[-2] // block_rows), -(-shape[-1] // BLOCK))


def quantize(x, block_rows=1):
    """(codes uint8, scales fp32) of x [.., N, K] fp32 (or what fp32 holds)."""
    x = np.asarray(x, dtype=np.float32)
    codes = np.zeros(x.shape, np.uint8)
    scales = np.zeros(scale_shape(x.shape, block_rows), np.float32)
    for lead in np.ndindex(x.shape[:-2]):
        for i in range(scales.shape[-2]):
            for j in range(scales.shape[-1]):
                at = (*lead, slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK))
                b = x[at]
                if not np.isfinite(b).all():
                    scales[(*lead, i, j)] = np.nan
                    continue
                s = max(np.float32(np.abs(b).max()) / np.float32(448), np.float32(2.0 ** -126))
                scales[(*lead, i, j)] = s
                codes[at] = encode(b / s)   # fp32 / fp32: rounded once
    return codes, scales


def dequantize(codes, scales) -> np.ndarray:
    """The fp64 values [.., N, K] of codes and their scales (whose shape gives the rows of a block)."""
    codes, scales = np.asarray(codes), np.asarray(scales, dtype=np.float64)
    n, k = codes.shape[-2:]
    rows = 1 if scales.shape[-2] == n else BLOCK
    s = np.repeat(np.repeat(scales, rows, axis=-2)[..., :n, :], BLOCK, axis=-1)[..., :k]
    return decode(codes) * s


def forward(x, w) -> np.ndarray:
    """Y [M, N] = x w^T of two pairs (codes, scales), fp64."""
    return dequantize(*x) @ dequantize(*w).T


def grouped_forward(x, w, offsets, rows=None) -> np.ndarray:
    """fp64 Y [M, N] of the products grouped by expert; NaN in the rows that no expert owns."""
    xv = dequantize(*x)
    if rows is not None:
        xv = xv[np.asarray(rows)]
    wv = dequantize(*w)
    y = np.full((xv.shape[0], wv.shape[1]), np.nan)
    for e in range(wv.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = xv[lo:hi] @ wv[e].T
    return y
