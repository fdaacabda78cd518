"""MXFP4: E2M1 codes with one E8M0 factor per 32 elements, products and products grouped by expert.

Test infrastructure only (see the package docstring).  The element format is that of
``fp4``; the block factor is the microscaling formats' E8M0 byte s, 2^(s - 127), 255 = NaN.
"""
from __future__ import annotations

import math

import numpy as np

from .fp4 import e2m1_value
from .int4 import pack_nibbles, unpack_nibbles

BLOCK = 32


def e8m0_value(byte) -> np.ndarray:
    """fp64 value of E8M0 bytes."""
    b = np.asarray(byte).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.where(b == 255, 0, b - 127)))


def _code(y: float) -> int:
    """E2M1 code of y by the distance to every magnitude, ties to the even code."""
    mags = [float(v) for v in e2m1_value(np.arange(8))]
    a = min(abs(y), 6.0)
    best = min(range(8), key=lambda i: (abs(mags[i] - a), i & 1))
    return best | 8 if y < 0 and best else best


def quantize_scalar(block):
    """(32 codes, scale byte) of one block, one value at a time."""
    vals = [float(v) for v in block]
    if any(math.isnan(v) or math.isinf(v) for v in vals):
        return [0] * len(vals), 255
    a = max(abs(v) for v in vals)
    e = -127 if a == 0 else max(math.frexp(a)[1] - 1 - 2, -127)
    return [_code(math.ldexp(v, -e)) for v in vals], e + 127


def quantize(x):
    """(codes [M, K/2] uint8, scales [M, K/32] uint8) of x [M, K] (any float type, exactly widened)."""
    x = np.asarray(x, dtype=np.float64)
    m, k = x.shape
    if k % BLOCK:
        raise ValueError("K must be a multiple of 32")
    b = x.reshape(m, k // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    a = np.abs(b).max(axis=-1, initial=0.0)
    e = np.where(a == 0, -127, np.maximum(np.frexp(a)[1] - 3, -127))
    y = np.ldexp(b, -e[..., None])
    mags = e2m1_value(np.arange(8))
    dist = np.abs(np.minimum(np.abs(y), 6.0)[..., None] - mags)
    near = dist == dist.min(axis=-1, keepdims=True)
    # of two equally near codes (neighbours) the even one
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    code = np.where((y < 0) & (pick > 0), pick | 8, pick)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(m, k)
    return pack_nibbles(code), np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(codes, scales) -> np.ndarray:
    """The fp64 values [..., K] of codes [..., K/2] and scales [..., K/32]."""
    codes = np.asarray(codes)
    lead = codes.shape[:-1]
    c = unpack_nibbles(codes.reshape(-1, codes.shape[-1]))
    f = np.repeat(e8m0_value(np.asarray(scales).reshape(c.shape[0], -1)), BLOCK, axis=-1)
    return (e2m1_value(c) * f).reshape(*lead, -1)


def forward(x, codes, scales) -> np.ndarray:
    """Y [M, N] = x W^T, fp64."""
    return np.asarray(x, dtype=np.float64) @ dequantize(codes, scales).T


def grouped_forward(x, codes, scales, offsets, rows=None) -> np.ndarray:
    """fp64 Y [M, N] of the products grouped by expert; NaN in the rows that no expert owns."""
    x = np.asarray(x, dtype=np.float64)
    if rows is not None:
        x = x[np.asarray(rows)]
    y = np.full((x.shape[0], codes.shape[1]), np.nan)
    for e in range(codes.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = forward(x[lo:hi], codes[e], scales[e])
    return y
