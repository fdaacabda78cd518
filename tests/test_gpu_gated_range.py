"""The gated activation over the whole range of g: silu's error grows with |g|, and below -87.34 silu is a zero."""
import numpy as np
import pytest
import torch

from tests.gpu_util import dev, host, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_silu_from_lowest_to_highest():
    """One value of g a row, u so that h is of ordinary size: the block's scale is |h| / 448 and every code +-448, so reading
    back gives h within the scale's rounding, 2^-24, the product's, 2^-24, and silu's (2 |g| + 8) 2^-23."""
    from weight_only_bit_group_amd import binding as B
    g = np.concatenate([-np.geomspace(1e-30, 87.3, 400), np.geomspace(1e-30, 1e30, 400), [-87.336, 3e38, -1e-38, 0.0]]).astype(np.float32)
    silu = g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64)))
    u = np.where(silu == 0, 1.0, np.clip(1 / np.where(silu == 0, 1, np.abs(silu)), 1e-37, 1e37)).astype(np.float32)
    h = dev(np.concatenate([np.repeat(g[:, None], 128, 1), np.repeat(u[:, None], 128, 1)], 1))
    step("gated activation over the range of g")
    c, s = B.aq_fp8_swiglu_quantize(h)
    y = host(B.aq_fp8_dequantize(c, s).double())
    ref = silu * u
    assert (np.abs(y - ref[:, None]) <= (((2 * np.abs(np.clip(g, -100, 100)) + 8) * 2.0 ** -23 + 3 * 2.0 ** -24) * np.abs(ref))[:, None]).all()


def test_silu_below_the_normal_numbers_is_zero():
    from weight_only_bit_group_amd import binding as B
    g = np.array([-87.34, -88.0, -88.7, -89.0, -1e3, -1e30, np.finfo(np.float32).min], np.float32)
    h = dev(np.concatenate([np.repeat(g[:, None], 128, 1), np.full((len(g), 128), 1e30, np.float32)], 1))
    step("gated activation of the lowest g")
    c, s = B.aq_fp8_swiglu_quantize(h)
    assert (host(c.view(torch.uint8)) & 0x7F == 0).all() and (host(s) == 2.0 ** -126).all()
    h[:, :128] = float("-inf")
    c, s = B.aq_fp8_swiglu_quantize(h)
    assert s.isnan().all() and (c.view(torch.uint8) == 0).all()
