"""Refusals of the MXFP4 entry points (no GPU: validation precedes every launch) and of their binding."""
import pytest
import torch

from weight_only_bit_group_amd import _lib
from weight_only_bit_group_amd import binding as B

FAKE = 0x10000
BIG = 1 << 30


def _q(lib, X=FAKE, dt=1, M=4, K=64, ldx=None, C=FAKE, S=FAKE):
    return lib.aq_mxfp4_quantize(X, dt, M, K, K if ldx is None else ldx, C, S, None)


def _d(lib, C=FAKE, S=FAKE, M=4, K=64, Y=FAKE, dt=0):
    return lib.aq_mxfp4_dequantize(C, S, M, K, Y, dt, None)


def _g(lib, a4=False, X=FAKE, XS=FAKE, M=4, K=64, ldx=None, C=FAKE, S=FAKE, N=8, Y=FAKE, dt=0):
    if a4:
        return lib.aq_mxfp4_gemm_a4(X, XS, M, K, C, S, N, Y, dt, None)
    return lib.aq_mxfp4_gemm(X, M, K, K if ldx is None else ldx, C, S, N, Y, dt, None)


def _e(lib, a4=False, X=FAKE, XS=FAKE, T=4, K=64, ldx=None, C=FAKE, S=FAKE, E=2, N=8, off=FAKE, rows=None, M=4, Y=FAKE,
       dt=0):
    if a4:
        return lib.aq_mxfp4_grouped_gemm_a4(X, XS, T, K, C, S, E, N, off, rows, M, Y, dt, None)
    return lib.aq_mxfp4_grouped_gemm(X, T, K, K if ldx is None else ldx, C, S, E, N, off, rows, M, Y, dt, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dt=2), "dtype"), (dict(M=-1), "M"), (dict(M=BIG), "M"), (dict(K=48), "multiple of 32"), (dict(K=0), "K"),
    (dict(K=BIG), "K"), (dict(M=1 << 20, K=1 << 16), "2^36"), (dict(X=None), "X"), (dict(X=FAKE + 8), "aligned"),
    (dict(C=FAKE + 8), "codes"), (dict(C=None), "codes"), (dict(S=None), "scales"), (dict(ldx=32), "ldx"),
    (dict(ldx=68), "ldx"), (dict(dt=0, ldx=66), "ldx")])
def test_quantize_einval(lib, kw, frag):
    assert _q(lib, **kw) == _lib.AQ_EINVAL
    assert frag in _lib.last_error()


@pytest.mark.parametrize("kw", [dict(dt=5), dict(M=-1), dict(K=16), dict(C=None), dict(C=FAKE + 4), dict(S=None),
                                dict(Y=None), dict(Y=FAKE + 8), dict(M=1 << 20, K=1 << 16)])
def test_dequantize_einval(lib, kw):
    assert _d(lib, **kw) == _lib.AQ_EINVAL


COMMON = [dict(dt=2), dict(K=0), dict(K=48), dict(K=1 << 22), dict(N=-1), dict(N=1 << 22), dict(M=-1), dict(M=BIG),
          dict(X=None), dict(X=FAKE + 8), dict(C=None), dict(C=FAKE + 4), dict(S=None), dict(Y=None),
          dict(Y=FAKE + 4), dict(dt=1, Y=FAKE + 2)]


@pytest.mark.parametrize("kw", COMMON)
def test_products_einval(lib, kw):
    for call in (_g, _e):
        for a4 in (False, True):
            assert call(lib, a4, **kw) == _lib.AQ_EINVAL, (call, a4)


def test_products_einval_of_sizes_past_the_offsets(lib):
    """X's 16-byte units and the launch's threads are counted in 32 bits."""
    for a4, K in ((False, 1 << 11), (True, 1 << 13)):   # rows of 4 KiB
        for call, kw in ((_g, {}), (_e, dict(T=1 << 24))):
            assert call(lib, a4, M=1 << 24, K=K, **kw) == _lib.AQ_EINVAL and "2^36" in _lib.last_error()
        assert _e(lib, a4, T=1 << 24, K=K, M=4, rows=FAKE) == _lib.AQ_EINVAL and "2^36" in _lib.last_error()
        for call, kw in ((_g, {}), (_e, dict(T=1 << 20))):
            assert call(lib, a4, M=1 << 20, N=1 << 17, **kw) == _lib.AQ_EINVAL and "2^37" in _lib.last_error()
    assert _g(lib, False, M=1 << 18, K=64, ldx=1 << 17) == _lib.AQ_EINVAL and "2^36" in _lib.last_error()
    assert _e(lib, E=1 << 20, N=8) == _lib.AQ_EINVAL and "E out" in _lib.last_error()


def test_products_einval_of_one_kind(lib):
    for call in (_g, _e):
        assert call(lib, True, XS=None) == _lib.AQ_EINVAL and "x_scales" in _lib.last_error()
        for ldx in (56, 68, BIG):
            assert call(lib, False, ldx=ldx) == _lib.AQ_EINVAL and "ldx" in _lib.last_error()


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=-1), dict(E=BIG), dict(E=1 << 20, N=1 << 7), dict(T=-1),
                                dict(T=BIG, M=4), dict(T=3), dict(T=0, rows=FAKE), dict(off=None), dict(off=FAKE + 2),
                                dict(rows=FAKE + 2), dict(M=1 << 29, T=1 << 29, N=1 << 9)])
def test_grouped_einval(lib, kw):
    for a4 in (False, True):
        assert _e(lib, a4, **kw) == _lib.AQ_EINVAL, a4


def test_empty_calls_are_noops(lib):
    assert _q(lib, M=0) == _d(lib, M=0) == _lib.AQ_OK
    for a4 in (False, True):
        assert _g(lib, a4, M=0) == _g(lib, a4, N=0) == _lib.AQ_OK
        assert _e(lib, a4, M=0) == _e(lib, a4, N=0) == _e(lib, a4, M=0, T=0) == _lib.AQ_OK


def test_injected_runtime_failure(lib, monkeypatch):
    monkeypatch.setenv("AQ_FAULT_INJECT", "launch")
    assert _q(lib) == _d(lib) == _lib.AQ_ERUNTIME
    for a4 in (False, True):
        assert _g(lib, a4) == _e(lib, a4) == _lib.AQ_ERUNTIME
        assert "injected" in _lib.last_error()


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    for call in (lambda: B.aq_mxfp4_quantize(x), lambda: B.aq_mxfp4_dequantize(c, s), lambda: B.aq_mxfp4_gemm(x, c, s),
                 lambda: B.aq_mxfp4_gemm_a4(c, s, c, s),
                 lambda: B.aq_mxfp4_grouped_gemm(x, c[None], s[None], torch.zeros(2, dtype=torch.int32)),
                 lambda: B.aq_mxfp4_grouped_gemm_a4(c, s, c[None], s[None], torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        B.aq_mxfp4_quantize([1.0])
