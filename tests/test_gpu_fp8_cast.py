"""FP8 modules answer the same after the model around them was cast, moved, or loaded from the other type of codes."""
import copy

import pytest
import torch

from tests.gpu_util import step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _call(model):
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(33, 144, generator=g, device="cuda").bfloat16()
    ids, w = torch.randint(0, 5, (33, 2), generator=g, device="cuda"), torch.rand(33, 2, generator=g, device="cuda")
    return model["linear"](x), model["experts"](x, ids, w)


def _model():
    from weight_only_bit_group_amd import layer as L
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return torch.nn.ModuleDict({"linear": L.FP8Linear.from_weight(r(200, 144)), "experts": L.FP8Experts.from_weights(r(5, 128, 144), r(5, 144, 64)),
                                "other": torch.nn.Linear(8, 8, device="cuda")})


def _as(model, dtype):
    """The same modules with their codes as float8 or as bytes."""
    from weight_only_bit_group_amd import layer as L
    a, b = model["linear"], model["experts"]
    return torch.nn.ModuleDict({"linear": L.FP8Linear(a.codes.view(dtype), a.scales), "other": model["other"],
                                "experts": L.FP8Experts(b.gate_up_codes.view(dtype), b.gate_up_scales, b.down_codes.view(dtype), b.down_scales)})


def test_casts_moves_and_loads_keep_the_answers():
    model = _model()
    ref = _call(model)
    step("FP8 modules after casts, moves and loads")
    same = lambda m: all(torch.equal(a, b) for a, b in zip(_call(m), ref))
    for cast in (lambda m: m.to(torch.bfloat16), lambda m: m.half(), lambda m: m.double(), lambda m: m.half().cpu().float().cuda(),
                 lambda m: m.cpu().to("cuda", torch.bfloat16), lambda m: m.type(torch.float16)):
        assert same(cast(copy.deepcopy(model)))
    for have in (torch.float8_e4m3fn, torch.uint8):
        for given in (torch.float8_e4m3fn, torch.uint8):
            blank = copy.deepcopy(_as(model, have))
            for b in blank.buffers():
                b.zero_()
            blank.load_state_dict(_as(model, given).state_dict())
            assert same(blank) and blank["linear"].codes.dtype == have
