"""Refusals of the MXFP4 modules that need no GPU."""
import pytest
import torch

from weight_only_bit_group_amd import layer as L

U8 = torch.uint8


def _pair(*lead, k=64):
    return torch.zeros(*lead, k // 2, dtype=U8), torch.zeros(*lead, k // 32, dtype=U8)


def test_linear_refuses_wrong_buffers():
    c, s = _pair(8)
    L.MXFP4Linear(c, s)
    for bad in ((c.int(), s), (c, s.float()), (c[0], s), (c, s[:4]), (c[:, :24], s), (c[:, :0], s[:, :0]), (c, s, None, "fp8")):
        with pytest.raises(ValueError):
            L.MXFP4Linear(*bad)


def test_experts_refuse_wrong_buffers():
    gu, d = _pair(3, 128, k=96), _pair(3, 96, k=64)
    m = L.MXFP4Experts(*gu, *d)
    assert (m.num_experts, m.features, m.inner) == (3, 96, 64)
    for bad in ((*gu, *_pair(3, 64, k=64)), (*gu, *_pair(2, 96, k=64)), (*gu, *_pair(3, 96, k=96)), (*_pair(384, k=96), *d),
                (*gu, d[0], d[1][..., :1]), (*gu, *d, "int8")):
        with pytest.raises(ValueError):
            L.MXFP4Experts(*bad)


def test_quantized_linear_is_not_quantized_again():
    model = torch.nn.ModuleDict({"a": L.MXFP4Linear(*_pair(8)), "b": torch.nn.Linear(64, 8)})
    with pytest.raises(ValueError, match="already quantized: a"):
        L.plan_quantization(model, ("a", "b"))
    assert list(L.plan_quantization(model, ("b",))) == ["b"]
    with pytest.raises(ValueError, match="already quantized"):
        L.quantize_linear(model["a"], 64)


def test_weights_on_the_host_are_refused():
    with pytest.raises(ValueError, match="GPU tensor"):
        L.MXFP4Linear.from_weight(torch.zeros(8, 64))
    with pytest.raises(ValueError, match="3 dimensions"):
        L.MXFP4Experts.from_weights(torch.zeros(8, 64), torch.zeros(2, 64, 32))
