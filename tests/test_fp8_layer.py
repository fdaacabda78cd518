"""FP8 modules as torch modules: casts and moves of a model that holds them (no GPU)."""
import copy

import pytest
import torch

from weight_only_bit_group_amd import layer as L

F8 = torch.float8_e4m3fn


def _pair(*lead, k=64):
    """Codes of every byte and scales that bf16 and fp16 do not hold."""
    g = torch.Generator().manual_seed(sum(lead) + k)
    codes = torch.randint(0, 256, (*lead, k), generator=g, dtype=torch.uint8)
    scales = torch.rand(*lead[:-1], -(-lead[-1] // 128), -(-k // 128), generator=g) + 1e-6
    return codes, scales


def _modules(codes_type=F8):
    c, s = _pair(200, k=272)
    linear = L.FP8Linear(c.view(codes_type), s, torch.arange(200.0))
    (gc, gs), (dc, ds) = _pair(3, 128, k=96), _pair(3, 96, k=64)
    return {"linear": linear, "experts": L.FP8Experts(gc.view(codes_type), gs, dc.view(codes_type), ds)}


def _held(model):
    """The codes' and scales' types and bytes, by name."""
    return {n: (b.dtype, b.contiguous().view(torch.uint8).clone()) for n, b in model.named_buffers() if not n.endswith("bias")}


def _unchanged(model, before):
    now = _held(model)
    assert now.keys() == before.keys()
    for n, (dtype, b) in before.items():
        assert now[n][0] == dtype and torch.equal(now[n][1], b), n


CASTS = {"to(bfloat16)": lambda m: m.to(torch.bfloat16), "half()": lambda m: m.half(), "float()": lambda m: m.float(),
         "double()": lambda m: m.double(), "to(device, dtype)": lambda m: m.to("cpu", torch.float16), "type": lambda m: m.type(torch.bfloat16),
         "to(tensor)": lambda m: m.to(torch.zeros(1, dtype=torch.bfloat16)), "to(float8)": lambda m: m.to(F8),
         "to(memory_format)": lambda m: m.to(memory_format=torch.contiguous_format), "cpu()": lambda m: m.cpu(),
         "share_memory": lambda m: m.share_memory(), "deepcopy": copy.deepcopy}


@pytest.mark.parametrize("codes_type", [F8, torch.uint8])
@pytest.mark.parametrize("cast", list(CASTS))
def test_casts_leave_codes_and_scales(cast, codes_type):
    """A cast of the model around the modules: codes and scales count as floating point, but their bits are the weights."""
    model = torch.nn.ModuleDict(_modules(codes_type) | {"other": torch.nn.Linear(8, 8)})
    before = _held(model)
    assert len(before) == 6
    model = CASTS[cast](model)
    _unchanged(model, before)
    if cast in ("to(bfloat16)", "type", "to(tensor)"):
        assert model["other"].weight.dtype == model["linear"].bias.dtype == torch.bfloat16


def test_casts_move_codes_and_scales():
    for name, m in _modules().items():
        types = [b.dtype for b in m.buffers()]
        for moved in (copy.deepcopy(m).to("meta", torch.bfloat16), copy.deepcopy(m).to("meta"), copy.deepcopy(m).to_empty(device="meta")):
            assert all(b.is_meta for b in moved.buffers()) and len(list(moved.buffers())) == len(types)
            assert [b.dtype for n, b in moved.named_buffers() if n != "bias"] == [b.dtype for n, b in m.named_buffers() if n != "bias"], name
