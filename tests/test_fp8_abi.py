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


def _g(lib, X=FAKE, XS=FAKE, M=4, K=64, C=FAKE, S=FAKE, N=8, Y=FAKE, dt=0):
    return lib.aq_fp8_gemm(X, XS, M, K, C, S, N, Y, dt, None)


def _l(lib, X=FAKE, xdt=1, M=4, K=64, ldx=None, C=FAKE, S=FAKE, N=8, Y=FAKE, dt=0, W=FAKE, wb=None):
    return lib.aq_fp8_linear(X, xdt, M, K, K if ldx is None else ldx, C, S, N, Y, dt, W, 1 << 40 if wb is None else wb, None)


def _e(lib, X=FAKE, XS=FAKE, T=4, K=64, C=FAKE, S=FAKE, E=2, N=8, off=FAKE, rows=None, M=4, Y=FAKE, dt=0):
    return lib.aq_fp8_grouped_gemm(X, XS, T, K, C, S, E, N, off, rows, M, Y, dt, None)


@pytest.mark.parametrize("kw", [dict(dt=2), dict(K=0), dict(K=40), dict(K=1 << 22), dict(N=-1), dict(N=1 << 22), dict(M=-1),
                                dict(M=BIG), dict(X=None), dict(X=FAKE + 8), dict(C=None), dict(C=FAKE + 4), dict(S=None),
                                dict(S=FAKE + 2), dict(Y=None), dict(Y=FAKE + 2), dict(dt=1, Y=FAKE + 1)])
def test_products_einval(lib, kw):
    for call in (_g, _l, _e):
        assert call(lib, **kw) == _lib.AQ_EINVAL, call


def test_products_einval_of_sizes_past_the_offsets(lib):
    for call, kw in ((_g, {}), (_l, {}), (_e, dict(T=1 << 24))):
        assert call(lib, M=1 << 24, K=1 << 12, **kw) == _lib.AQ_EINVAL and "2^36" in _lib.last_error()
    for call, kw in ((_g, {}), (_l, {}), (_e, dict(T=1 << 20))):
        assert call(lib, M=1 << 20, N=1 << 17, **kw) == _lib.AQ_EINVAL and "2^37" in _lib.last_error()


@pytest.mark.parametrize("kw,frag", [(dict(xdt=3), "x_dtype"), (dict(ldx=56), "ldx"), (dict(ldx=68), "ldx"), (dict(W=None), "workspace"),
                                     (dict(W=FAKE + 8), "workspace"), (dict(wb=4 * 64 + 15), "workspace")])
def test_linear_einval(lib, kw, frag):
    assert _l(lib, **kw) == _lib.AQ_EINVAL and frag in _lib.last_error()


def test_linear_workspace(lib):
    assert lib.aq_fp8_linear_workspace(4, 64) == 4 * 64 + 16 and lib.aq_fp8_linear_workspace(3, 272) == 3 * (272 + 12)
    assert lib.aq_fp8_linear_workspace(0, 64) == lib.aq_fp8_linear_workspace(4, 40) == lib.aq_fp8_linear_workspace(-1, 64) == 0


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=-1), dict(E=1 << 20), dict(E=1 << 19, N=1 << 8), dict(T=-1), dict(T=BIG, M=4),
                                dict(T=3), dict(T=0, rows=FAKE), dict(off=None), dict(off=FAKE + 2), dict(rows=FAKE + 2),
                                dict(XS=None), dict(XS=FAKE + 1)])
def test_grouped_einval(lib, kw):
    assert _e(lib, **kw) == _lib.AQ_EINVAL


def test_empty_products_and_injected_failures(lib, monkeypatch):
    assert _g(lib, M=0) == _g(lib, N=0) == _l(lib, N=0) == _l(lib, M=0, W=None) == _e(lib, M=0, T=0) == _e(lib, N=0) == _lib.AQ_OK
    monkeypatch.setenv("AQ_FAULT_INJECT", "launch")
    assert _g(lib) == _l(lib) == _e(lib) == _lib.AQ_ERUNTIME


def test_binding_products_refuse_host_tensors():
    c, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    w, ws = torch.zeros(8, 64, dtype=torch.float8_e4m3fn), torch.zeros(1, 1)
    for call in (lambda: B.aq_fp8_gemm(c, s, w, ws), lambda: B.aq_fp8_linear(c.float(), w, ws),
                 lambda: B.aq_fp8_grouped_gemm(c, s, w[None], ws[None], torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
