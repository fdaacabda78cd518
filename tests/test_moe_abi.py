"""Refusals of the routing entry points and of the FP8 modules (no GPU: validation precedes every launch)."""
import pytest
import torch

from weight_only_bit_group_amd import _lib
from weight_only_bit_group_amd import binding as B
from weight_only_bit_group_amd import layer as L

FAKE = 0x10000
BIG = 1 << 30
F8 = torch.float8_e4m3fn


def _r(lib, L=FAKE, dt=0, T=4, E=8, ld=None, top=2, score=0, bias=None, G=1, TG=1, rn=1, sc=1.0, I=FAKE, W=FAKE):
    return lib.aq_moe_route(L, dt, T, E, E if ld is None else ld, top, score, bias, G, TG, rn, sc, I, W, None)


def _b(lib, L=FAKE, dt=0, T=4, E=8, ld=None, top=2, score=0, rn=1, sc=1.0, I=FAKE, W=FAKE, D=FAKE, DL=FAKE):
    return lib.aq_moe_route_backward(L, dt, T, E, E if ld is None else ld, top, score, rn, sc, I, W, D, DL, None)


COMMON = [dict(dt=2), dict(score=2), dict(T=-1), dict(T=BIG), dict(E=0), dict(E=1025), dict(top=0), dict(top=9), dict(E=128, top=65),
          dict(ld=7), dict(ld=BIG), dict(sc=float("inf")), dict(sc=float("nan")), dict(L=None), dict(L=FAKE + 2), dict(I=None),
          dict(I=FAKE + 2), dict(W=None), dict(W=FAKE + 1), dict(dt=1, L=FAKE + 1)]


@pytest.mark.parametrize("kw", COMMON)
def test_route_einval(lib, kw):
    assert _r(lib, **kw) == _lib.AQ_EINVAL and _b(lib, **kw) == _lib.AQ_EINVAL


@pytest.mark.parametrize("kw,frag", [(dict(G=0), "groups"), (dict(G=3), "groups"), (dict(E=128, G=128), "groups"), (dict(G=4, TG=0), "top_groups"),
                                     (dict(G=4, TG=5), "top_groups"), (dict(G=4, TG=1, top=3), "top_groups"), (dict(bias=FAKE + 2), "bias")])
def test_groups_einval(lib, kw, frag):
    assert _r(lib, **kw) == _lib.AQ_EINVAL and frag in _lib.last_error()


@pytest.mark.parametrize("kw", [dict(D=None), dict(D=FAKE + 2), dict(DL=None), dict(DL=FAKE + 2)])
def test_backward_einval(lib, kw):
    assert _b(lib, **kw) == _lib.AQ_EINVAL


def _g(lib, I=FAKE, T=4, top=2, E=8, O=FAKE, R=FAKE, S=FAKE, W=None, wb=0):
    return lib.aq_moe_group(I, T, top, E, O, R, S, W, wb, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=BIG), dict(top=0), dict(T=1 << 29, top=4), dict(E=0), dict(E=1025), dict(I=None),
                                dict(O=None), dict(R=None), dict(S=None), dict(I=FAKE + 2), dict(O=FAKE + 2), dict(R=FAKE + 1),
                                dict(S=FAKE + 2), dict(T=1 << 14, W=FAKE), dict(T=1 << 14, wb=BIG), dict(T=1 << 14, W=FAKE + 2, wb=BIG)])
def test_group_einval(lib, kw):
    assert _g(lib, **kw) == _lib.AQ_EINVAL


def test_group_workspace(lib):
    assert lib.aq_moe_group_workspace(1 << 13, 2, 8) == 0 and lib.aq_moe_group_workspace(1 << 13, 3, 8) == 6 * 8 * 4
    assert lib.aq_moe_group_workspace(-1, 2, 8) == lib.aq_moe_group_workspace(1 << 20, 2, 2000) == 0


def _c(lib, Y=FAKE, ydt=0, R=8, K=64, S=FAKE, W=FAKE, T=4, top=2, O=FAKE, dt=0):
    return lib.aq_moe_combine(Y, ydt, R, K, S, W, T, top, O, dt, None)


def _cb(lib, Y=FAKE, ydt=0, R=8, K=64, S=FAKE, W=FAKE, T=4, top=2, O=FAKE, dt=0):
    return lib.aq_moe_combine_backward(Y, ydt, R, K, S, T, top, O, dt, W, None)


@pytest.mark.parametrize("kw", [dict(ydt=2), dict(dt=3), dict(T=-1), dict(T=BIG), dict(top=0), dict(T=1 << 29, top=4), dict(R=-1), dict(R=0),
                                dict(R=1 << 31), dict(K=0), dict(K=12), dict(K=1 << 22), dict(T=1 << 26, K=1 << 10), dict(Y=None), dict(Y=FAKE + 8),
                                dict(S=None), dict(S=FAKE + 2), dict(W=None), dict(W=FAKE + 2), dict(O=None), dict(O=FAKE + 8)])
def test_combine_einval(lib, kw):
    assert _c(lib, **kw) == _lib.AQ_EINVAL and _cb(lib, **kw) == _lib.AQ_EINVAL


def _s(lib, H=FAKE, dt=0, M=4, I=64, end=None, C=FAKE, S=FAKE):
    return lib.aq_fp8_swiglu_quantize(H, dt, M, I, end, C, S, None)


@pytest.mark.parametrize("kw", [dict(dt=2), dict(M=-1), dict(M=BIG), dict(I=0), dict(I=24), dict(I=1 << 22), dict(M=1 << 20, I=1 << 16),
                                dict(H=None), dict(H=FAKE + 8), dict(C=None), dict(C=FAKE + 8), dict(S=None), dict(S=FAKE + 2),
                                dict(end=FAKE + 2)])
def test_swiglu_einval(lib, kw):
    assert _s(lib, **kw) == _lib.AQ_EINVAL


def test_empty_calls_and_injected_failures(lib, monkeypatch):
    assert _r(lib, T=0) == _b(lib, T=0) == _c(lib, T=0, R=0) == _cb(lib, T=0) == _s(lib, M=0) == _lib.AQ_OK
    monkeypatch.setenv("AQ_FAULT_INJECT", "launch")
    assert _r(lib) == _b(lib) == _g(lib) == _c(lib) == _cb(lib) == _s(lib) == _lib.AQ_ERUNTIME


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: B.aq_moe_route(x, 2), lambda: B.aq_moe_route_backward(x, i, i.float(), i.float()), lambda: B.aq_moe_group(i, 8),
                 lambda: B.aq_moe_combine(x, i, i.float()), lambda: B.aq_moe_combine_backward(x, i, x), lambda: L.route(x, 2),
                 lambda: B.aq_fp8_swiglu_quantize(torch.zeros(4, 64))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: B.aq_moe_route([1.0], 2), lambda: B.aq_moe_group([1], 8), lambda: B.aq_moe_combine([1.0], i, i.float())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="score"):
        B._score("tanh")


def _pair(*lead, k=64):
    return torch.zeros(*lead, k, dtype=F8), torch.zeros(*lead[:-1], -(-lead[-1] // 128), -(-k // 128))


def test_linear_refuses_wrong_buffers():
    c, s = _pair(200, k=272)
    assert L.FP8Linear(c, s).in_features == 272 and L.FP8Linear(c.view(torch.uint8), s).out_features == 200
    for bad in ((c.float(), s), (c, s.double()), (c[0], s), (c, s[:1]), (c[:, :264], s), (c[:, :0], s[:, :0]), (c, s, None, torch.float16)):
        with pytest.raises(ValueError):
            L.FP8Linear(*bad)
    with pytest.raises(ValueError, match="input features"):
        L.FP8Linear(c, s)(torch.zeros(3, 256))
    with pytest.raises(ValueError, match="GPU tensor"):
        L.FP8Linear.from_weight(torch.zeros(8, 64))


def test_experts_refuse_wrong_buffers_and_choices():
    gu, d = _pair(3, 128, k=96), _pair(3, 96, k=64)
    m = L.FP8Experts(*gu, *d)
    assert (m.num_experts, m.features, m.inner) == (3, 96, 64)
    for bad in ((*gu, *_pair(3, 64, k=64)), (*gu, *_pair(2, 96, k=64)), (*gu, *_pair(3, 96, k=96)), (*gu, d[0], d[1][:, :0]),
                (*gu, *d, torch.float16), (*_pair(1025, 32, k=16), *_pair(1025, 16, k=16))):
        with pytest.raises(ValueError):
            L.FP8Experts(*bad)
    x, i = torch.zeros(4, 96), torch.zeros(4, 2, dtype=torch.int32)
    for bad in ((x[:, :64], i, i.float()), (x, i, i.float()[:, :1]), (x, i[:3], i[:3].float()), (x, i.float(), i.float()),
                (x, i.bool(), i.float()), (x, i[:, :0], i[:, :0].float())):
        with pytest.raises(ValueError):
            m(*bad)


def test_quantized_linear_is_not_quantized_again():
    model = torch.nn.ModuleDict({"a": L.FP8Linear(*_pair(8)), "b": torch.nn.Linear(64, 8)})
    with pytest.raises(ValueError, match="already quantized: a"):
        L.plan_quantization(model, ("a", "b"))
    with pytest.raises(ValueError, match="already quantized"):
        L.quantize_linear(model["a"], 64)
