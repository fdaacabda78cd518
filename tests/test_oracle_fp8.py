"""Pins of the FP8 oracle: the E4M3 values, the rounding against brute force, closed forms of the block scale, and
the grouped product against the plain one."""
import numpy as np
import pytest

from oracle import fp8


def test_values():
    v = fp8.decode(np.arange(256))
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0xB8] == -1.0
    assert np.isnan(v[[0x7F, 0xFF]]).all() and (np.diff(v[:127]) > 0).all()


def test_encode_is_the_nearest_code():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.standard_normal(2000) * np.exp(rng.uniform(-8, 5, 2000)), fp8.decode(np.arange(127)),
                        -fp8._MIDS, fp8._MIDS, np.nextafter(fp8._MIDS, 0), np.nextafter(fp8._MIDS, 500), [463.9, -0.0]])
    y = y[np.abs(y) < 464]
    assert fp8.encode(y).tolist() == [fp8.encode_scalar(float(v)) for v in y]
    assert fp8.encode(np.float64(-0.0)) == 128 and fp8.encode(np.float64(-1e-9)) == 128
    assert (fp8.encode(fp8._MIDS) % 2 == 0).all()


def test_scales():
    x = np.zeros((1, 128), np.float32)
    assert fp8.quantize(x)[1][0, 0] == np.float32(2.0 ** -126)
    for a, s in ((448.0, 1.0), (1.0, np.float32(1) / np.float32(448)), (1e-40, 2.0 ** -126), (3e38, np.float32(3e38) / np.float32(448))):
        x[0, 7] = -a
        c, got = fp8.quantize(x)
        assert got[0, 0] == np.float32(s)
        if a >= 1:
            assert c[0, 7] == 0xFE
    x[0, 3] = np.nan
    c, s = fp8.quantize(x)
    assert np.isnan(s).all() and (c == 0).all()


@pytest.mark.parametrize("shape", [(5, 48), (3, 130 * 16 // 16 * 16), (2, 200, 272), (129, 16), (1, 128, 128)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_values_lie_within_half_a_step(shape, block_rows):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(shape) * 3).astype(np.float32)
    c, s = fp8.quantize(x, block_rows)
    assert s.shape == fp8.scale_shape(shape, block_rows)
    w = fp8.dequantize(c, s)
    big = np.repeat(np.repeat(s.astype(np.float64), block_rows, -2)[..., :shape[-2], :], 128, -1)[..., :shape[-1]]
    assert (np.abs(w - x) <= np.maximum(np.abs(x) * 2.0 ** -4, big * 2.0 ** -10) * (1 + 2.0 ** -20)).all()


def test_grouped_forward():
    rng = np.random.default_rng(2)
    x = fp8.quantize(rng.standard_normal((6, 144)).astype(np.float32))
    w = fp8.quantize(rng.standard_normal((3, 130, 144)).astype(np.float32), 128)
    y = fp8.grouped_forward(x, w, [1, 3, 3, 5], [5, 0, 2, 2, 1, 3])
    for r, (e, t) in enumerate([(None, 5), (0, 0), (0, 2), (2, 2), (2, 1), (None, 3)]):
        if e is None:
            assert np.isnan(y[r]).all()
        else:
            one = fp8.forward((x[0][t:t + 1], x[1][t:t + 1]), (w[0][e], w[1][e]))[0]
            assert np.allclose(y[r], one, rtol=1e-13, atol=1e-13 * np.abs(one).max())
