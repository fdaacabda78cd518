"""Refusals of the FP8 entry points (no GPU: validation precedes every launch) and of their binding."""
import pytest
import torch

from weight_only_bit_group_amd import _lib
from weight_only_bit_group_amd import binding as B

FAKE = 0x10000
BIG = 1 << 30


def _q(lib, X=FAKE, dt=1, E=1, N=4, K=64, ldx=None, br=1, C=FAKE, S=FAKE):
    return lib.aq_fp8_quantize(X, dt, E, N, K, K if ldx is None else ldx, br, C, S, None)


def _d(lib, C=FAKE, S=FAKE, E=1, N=4, K=64, br=1, Y=FAKE, dt=0):
    return lib.aq_fp8_dequantize(C, S, E, N, K, br, Y, dt, None)


MATRIX = [dict(dt=2), dict(E=0), dict(E=-1), dict(N=-1), dict(N=BIG), dict(E=1 << 20, N=1 << 10), dict(K=0), dict(K=24),
          dict(K=BIG), dict(N=1 << 20, K=1 << 16), dict(br=0), dict(br=64), dict(C=None), dict(C=FAKE + 8), dict(S=None),
          dict(S=FAKE + 2)]


@pytest.mark.parametrize("kw", MATRIX)
def test_matrix_einval(lib, kw):
    assert _q(lib, **kw) == _lib.AQ_EINVAL
    assert _d(lib, **kw) == _lib.AQ_EINVAL


@pytest.mark.parametrize("kw,frag", [(dict(X=None), "X"), (dict(X=FAKE + 8), "aligned"), (dict(ldx=48), "ldx"),
                                     (dict(ldx=68), "ldx"), (dict(dt=0, ldx=66), "ldx"), (dict(K=40), "multiple of 16")])
def test_quantize_einval(lib, kw, frag):
    assert _q(lib, **kw) == _lib.AQ_EINVAL
    assert frag in _lib.last_error()


@pytest.mark.parametrize("kw", [dict(Y=None), dict(Y=FAKE + 8)])
def test_dequantize_einval(lib, kw):
    assert _d(lib, **kw) == _lib.AQ_EINVAL


def test_empty_calls_are_noops(lib):
    for br in (1, 128):
        assert _q(lib, N=0, br=br) == _d(lib, N=0, br=br) == _lib.AQ_OK


def test_injected_runtime_failure(lib, monkeypatch):
    monkeypatch.setenv("AQ_FAULT_INJECT", "launch")
    assert _q(lib) == _d(lib) == _lib.AQ_ERUNTIME
    assert "injected" in _lib.last_error()


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    for call in (lambda: B.aq_fp8_quantize(x), lambda: B.aq_fp8_dequantize(c, s)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        B.aq_fp8_quantize([1.0])
    with pytest.raises(ValueError, match="block_rows"):
        B._f8_scales((4, 64), 16)
