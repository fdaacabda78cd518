"""Pins of the MXFP4 oracle: the E8M0 values, the rounding against brute force over every code, closed forms of
the block exponent, and the grouped product against the plain one."""
import math

import numpy as np
import pytest

from oracle import fp4, mxfp4


def test_e8m0_values():
    v = mxfp4.e8m0_value(np.arange(256))
    assert v[127] == 1.0 and v[0] == 2.0 ** -127 and v[254] == 2.0 ** 127 and np.isnan(v[255])
    assert (v[1:255] / v[:254] == 2.0).all()


def test_block_exponent_closed_forms():
    for a, e in ((1.0, -2), (1.999, -2), (2.0, -1), (6.0, 0), (7.99, 0), (8.0, 1), (2.0 ** -130, -127), (0.0, -127),
                 (3.3e38, 125)):
        x = np.zeros((1, 32))
        x[0, 5] = -a
        assert mxfp4.quantize(x)[1][0, 0] == e + 127, a
    c, s = mxfp4.quantize(np.zeros((2, 64)))
    assert (c == 0).all() and (s == 0).all()


def test_codes_are_the_nearest_grid_points():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 96)) * np.exp(rng.standard_normal((40, 1)) * 8)).astype(np.float32)
    c, s = mxfp4.quantize(x)
    w = mxfp4.dequantize(c, s)
    grid = fp4.e2m1_value(np.arange(16))
    f = np.repeat(mxfp4.e8m0_value(s), 32, axis=-1)
    best = np.abs(x[..., None].astype(np.float64) - grid * f[..., None]).min(-1)
    assert (np.abs(w - x) == best).all()
    # the largest magnitude of a block lands in [4, 8) steps: its relative error is at most a quarter
    assert (np.abs(w - x) <= np.maximum(0.25 * np.abs(x), 0.5 * f * (1 + (np.abs(x) >= 4 * f)))).all()


def test_ties_go_to_even_codes_and_saturate():
    x = np.zeros((1, 32))
    x[0, :12] = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9, -.25, -5.0, -.75]
    c, s = mxfp4.quantize(x)
    assert s[0, 0] == 127
    assert mxfp4.dequantize(c, s)[0, :12].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6, 0, -4, -1]
    assert (c[0, 4] >> 4) == 0   # no sign on a zero magnitude


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_blocks_that_are_not_finite(bad):
    x = np.ones((1, 64))
    x[0, 40] = bad
    c, s = mxfp4.quantize(x)
    assert s[0].tolist() == [125, 255] and (c[0, 16:] == 0).all()
    assert np.isnan(mxfp4.dequantize(c, s)[0, 32:]).all()


def test_vector_form_equals_scalar_form():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 64)) * 3
    x[0, :32] = np.round(x[0, :32] * 4) / 4
    x[1, 3] = np.nan
    c, s = mxfp4.quantize(x)
    for i in range(6):
        for b in range(2):
            code, byte = mxfp4.quantize_scalar(x[i, 32 * b:32 * b + 32])
            got = c[i, 16 * b:16 * b + 16]
            assert byte == s[i, b] and code == [int(v) for p in got for v in (p & 15, p >> 4)]


def test_forward_by_loops_and_grouped_by_slices():
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 256, (3, 5, 32), dtype=np.uint8)
    scales = rng.integers(120, 134, (3, 5, 2), dtype=np.uint8)
    x = rng.standard_normal((7, 64))
    y = mxfp4.forward(x, codes[1], scales[1])
    for m in range(7):
        for n in range(5):
            want = 0.0
            for k in range(64):
                b = int(codes[1, n, k // 2])
                v = float(fp4.e2m1_value((b >> 4) if k & 1 else (b & 15)))
                want += x[m, k] * v * 2.0 ** (int(scales[1, n, k // 32]) - 127)
            assert abs(y[m, n] - want) <= 64 * 2.0 ** -52 * 6 * 2 ** 7 * 64
    rows = [4, 0, 6, 6, 1]
    g = mxfp4.grouped_forward(x, codes, scales, [1, 3, 3, 5], rows)
    assert np.isnan(g[0]).all()
    assert (g[1:3] == mxfp4.forward(x[[0, 6]], codes[0], scales[0])).all()
    assert (g[3:5] == mxfp4.forward(x[[6, 1]], codes[2], scales[2])).all()
