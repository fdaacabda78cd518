"""Refusals of the experts' call (no GPU: validation precedes every launch)."""
import pytest
import torch

from weight_only_bit_group_amd import _lib
from weight_only_bit_group_amd import binding as B

FAKE = 0x10000
BIG = 1 << 40


def _x(lib, X=FAKE, xdt=1, T=4, K=256, ldx=None, G=FAKE, GS=FAKE, D=FAKE, DS=FAKE, E=8, I=128, ids=FAKE, W=FAKE, top=2, P=FAKE, S=FAKE, O=FAKE,
       dt=1, work=FAKE, wb=BIG):
    return lib.aq_fp8_experts(X, xdt, T, K, K if ldx is None else ldx, G, GS, D, DS, E, I, ids, W, top, P, S, O, dt, work, wb, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(xdt=2), "x_dtype"), (dict(dt=2), "out_dtype"), (dict(T=-1), "T "), (dict(T=1 << 30), "T "), (dict(E=0), "E "), (dict(E=1025), "E "),
    (dict(top=0), "top"), (dict(T=1 << 29, top=4), "top"), (dict(T=1 << 29, top=2), "too large"), (dict(K=0), "K "), (dict(K=24), "K "),
    (dict(K=1 << 22), "K "), (dict(I=0), "I "), (dict(I=136), "I "), (dict(I=1 << 21), "I "), (dict(E=1024, I=1 << 17), "too large"),
    (dict(E=1024, K=1 << 17), "too large"), (dict(T=1 << 24, K=1 << 12), "too large"), (dict(T=1 << 23, top=8, I=1 << 10), "too large"),
    (dict(T=1 << 24, top=8, K=1 << 10), "too large"), (dict(ldx=248), "ldx"), (dict(ldx=260), "ldx"), (dict(xdt=0, ldx=258), "ldx"),
    (dict(G=None), "gate_up"), (dict(G=FAKE + 8), "gate_up"), (dict(GS=FAKE + 2), "gate_up_scales"), (dict(D=None), "down"),
    (dict(DS=None), "down_scales"), (dict(X=FAKE + 8), "X"), (dict(X=None), "X"), (dict(ids=None), "ids"), (dict(ids=FAKE + 2), "ids"),
    (dict(W=None), "weights"), (dict(P=FAKE + 8), "products"), (dict(P=None), "products"), (dict(S=FAKE + 1), "slots"), (dict(O=None), "out"),
    (dict(O=FAKE + 2), "out"), (dict(work=None), "workspace"), (dict(work=FAKE + 8), "workspace"), (dict(wb=1000), "workspace")])
def test_einval(lib, kw, frag):
    assert _x(lib, **kw) == _lib.AQ_EINVAL and frag in _lib.last_error()


def test_no_tokens_launch_nothing(lib):
    assert _x(lib, T=0, X=None, ids=None, W=None, P=None, S=None, O=None, work=None, wb=0) == _lib.AQ_OK


def test_injected_failure(lib, monkeypatch):
    monkeypatch.setenv("AQ_FAULT_INJECT", "launch")
    assert _x(lib) == _lib.AQ_ERUNTIME and "aq_fp8_experts" in _lib.last_error()


def test_workspace(lib):
    f = lib.aq_fp8_experts_workspace
    # lists, codes and scales of x and h, each on 256 bytes, and rows of [g | u] where the activation is a kernel of its own
    up = lambda n: -(-n // 256) * 256
    t, top, k, e, i = 5, 3, 272, 9, 144
    base = up(4 * (e + 1)) + up(4 * t * top) + up(t * k) + up(4 * t * 3) + up(t * top * i) + up(4 * t * top * 2)
    assert f(t, top, k, e, i) == base + up(8 * t * top * i)
    assert f(2048, 8, 2048, 64, 1408) < f(2048, 8, 2048, 64, 1424) - 16384 * 2 * 1408 * 4
    for bad in ((0, 2, 64, 8, 64), (-1, 2, 64, 8, 64), (4, 0, 64, 8, 64), (4, 2, 60, 8, 64), (4, 2, 64, 0, 64), (4, 2, 64, 2000, 64), (4, 2, 64, 8, 8)):
        assert f(*bad) == 0
    assert f(1 << 40, 1 << 40, 1 << 40, 1 << 40, 1 << 40) == 0


def test_binding_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.aq_fp8_experts(x, x, x, x, x, x, x)
