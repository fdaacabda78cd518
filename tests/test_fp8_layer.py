"""FP8 modules as torch modules: casts and moves of a model that holds them (no GPU)."""
import copy

import pytest
import torch
import torch.autograd.forward_ad as fw

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


@pytest.mark.parametrize("assign", [False, True])
@pytest.mark.parametrize("have", [F8, torch.uint8])
@pytest.mark.parametrize("given", [F8, torch.uint8])
def test_state_of_the_same_bytes_is_loaded_as_they_are(have, given, assign):
    """A checkpoint that holds the codes as bytes, into a module that holds them as float8, and the other way round."""
    whole = torch.nn.ModuleDict(_modules(given))
    blank = torch.nn.ModuleDict(_modules(have))
    before = {n: (dtype if dtype == torch.float32 else have, b) for n, (dtype, b) in _held(whole).items()}
    for m in blank.modules():
        for b in m.buffers(recurse=False):
            b.zero_()
    state = whole.state_dict()
    types = {n: t.dtype for n, t in state.items()}
    blank.load_state_dict(state, assign=assign)
    assert {n: t.dtype for n, t in state.items()} == types   # (the caller's own dict is left as it was)
    _unchanged(blank, before)
    assert torch.equal(blank["linear"].bias, whole["linear"].bias)


@pytest.mark.parametrize("assign", [False, True])
def test_state_of_another_kind_is_refused(assign):
    for name, m in _modules().items():
        codes = m._held[0]
        for dtype in (torch.bfloat16, torch.float32, torch.int8, torch.float8_e5m2, torch.float8_e4m3fnuz):
            state = m.state_dict()
            state[codes] = torch.zeros(state[codes].shape, dtype=dtype)
            before = _held(m)
            with pytest.raises(RuntimeError, match="float8_e4m3fn"):
                copy.deepcopy(m).load_state_dict(state, assign=assign)
            _unchanged(m, before)
        for dtype in (torch.bfloat16, torch.float64):   # (values that fp32 holds)
            state = m.state_dict()
            state[m._held[1]] = torch.full_like(state[m._held[1]], 0.75, dtype=dtype)
            other = copy.deepcopy(m)
            other.load_state_dict(state, assign=assign)
            scales = getattr(other, m._held[1])
            assert scales.dtype == torch.float32 and (scales == 0.75).all()
        state = m.state_dict()
        del state[codes]
        assert copy.deepcopy(m).load_state_dict(state, strict=False).missing_keys == [codes]


def test_inputs_with_a_tangent_are_refused():
    """A forward derivative is an error before anything else is looked at; without one the call goes on (to the binding, which
    wants a GPU tensor)."""
    m = _modules()
    ids = torch.zeros(4, 2, dtype=torch.int64)
    mx = L.MXFP4Linear(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8))
    calls = {"FP8Linear": (m["linear"], torch.randn(4, 272)), "MXFP4Linear": (mx, torch.randn(4, 64)),
             "FP8Experts": (lambda x: m["experts"](x, ids, ids.float()), torch.randn(4, 96)),
             "FP8Experts weights": (lambda w: m["experts"](torch.zeros(4, 96), ids, w), torch.randn(4, 2)),
             "route": (lambda l: L.route(l, 2), torch.randn(4, 8))}
    with fw.dual_level():
        for name, (call, x) in calls.items():
            for y in (x, x.double(), x.clone().requires_grad_()):
                with pytest.raises(RuntimeError, match=f"{name.split()[0]} has no forward derivative"):
                    call(fw.make_dual(y, torch.ones_like(y)))
            with pytest.raises(ValueError, match="GPU tensor"):
                call(x)
