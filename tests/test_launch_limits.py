"""The largest sizes that the routing and FP8 entry points accept are the largest that their launches can take (fewer than
2^32 threads); larger ones are refused before anything is launched.  (No GPU: with a failure injected in front of the
launch, a call whose arguments are accepted ends there.)"""
import pytest

from tests.test_fp8_abi import _d, _l, _q
from tests.test_fp8_experts_abi import _x
from tests.test_moe_abi import _b, _c, _cb, _g, _r, _s
from weight_only_bit_group_amd import _lib

BLOCKS = (1 << 24) - 1   # workgroups of 256 threads


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    monkeypatch.setenv("AQ_FAULT_INJECT", "launch")


def _limit(call, lib, inside, outside, frag):
    assert call(lib, **inside) == _lib.AQ_ERUNTIME and "injected" in _lib.last_error(), (call, inside)
    assert call(lib, **outside) == _lib.AQ_EINVAL and frag in _lib.last_error(), (call, outside)


@pytest.mark.parametrize("call", [_r, _b])
@pytest.mark.parametrize("E,top", [(1, 1), (8, 2), (64, 31)])
def test_tokens_of_route(lib, call, E, top):
    _limit(call, lib, dict(T=4 * BLOCKS, E=E, top=top), dict(T=4 * BLOCKS + 1, E=E, top=top), "T must be")


@pytest.mark.parametrize("K", [8, 64, 4096, (1 << 22) - 8])
def test_columns_of_combine(lib, K):
    t = 2048 * BLOCKS // K
    if t >= 1 << 30:
        assert _c(lib, T=(1 << 30) - 1, K=K, top=1) == _lib.AQ_ERUNTIME
    else:
        _limit(_c, lib, dict(T=t, K=K, top=1), dict(T=t + 1, K=K, top=1), "T * K")


@pytest.mark.parametrize("top", [1, 3, 8])
def test_choices_of_the_weighted_sums_gradient(lib, top):
    t = 4 * BLOCKS // top
    _limit(_cb, lib, dict(T=t, top=top, K=8), dict(T=t + 1, top=top, K=8), "T * top")
    assert _c(lib, T=t + 1, top=top, K=8) == _lib.AQ_ERUNTIME


@pytest.mark.parametrize("K", [16, 64])
def test_rows_of_the_quantiser(lib, K):
    """Of one block; longer rows end at 2^36 values before."""
    n = 64 * BLOCKS
    for call in (_q, _d):
        _limit(call, lib, dict(N=n, K=K), dict(N=n + 1, K=K), "blocks of 128")
        _limit(call, lib, dict(E=n // 4, N=4, K=K), dict(E=n // 4 + 1, N=4, K=K), "blocks of 128")
        assert call(lib, N=(1 << 36) // 144, K=144) == _lib.AQ_ERUNTIME
    _limit(_l, lib, dict(M=n, K=K), dict(M=n + 1, K=K), "blocks of 128")


@pytest.mark.parametrize("N", [1, 60, 63])
def test_blocks_of_the_quantiser(lib, N):
    """Many small matrices; of matrices of 128 rows and more 2^30 rows are fewer blocks."""
    _limit(_q, lib, dict(E=BLOCKS, N=N, K=16, br=128), dict(E=BLOCKS + 1, N=N, K=16, br=128), "128 x 128")
    _limit(_q, lib, dict(E=BLOCKS // 3, N=1, K=272, br=128), dict(E=BLOCKS // 3 + 1, N=1, K=272, br=128), "128 x 128")
    assert _d(lib, E=BLOCKS + 1, N=N, K=16, br=128) == _lib.AQ_ERUNTIME
    assert _q(lib, E=(1 << 23) - 1, N=128, K=16, br=128) == _lib.AQ_ERUNTIME


@pytest.mark.parametrize("I,blocks", [(16, 1), (128, 1), (144, 2), (208, 2)])
def test_blocks_of_the_gated_activation(lib, I, blocks):
    m = 16 * BLOCKS // blocks
    _limit(_s, lib, dict(M=m, I=I), dict(M=m + 1, I=I), "blocks of 128")


BIG = 1 << 60   # bytes of workspace


@pytest.mark.parametrize("inside,outside", [
    # the weighted sum, and few rows of K in blocks of 128 (2^35 - 2^21 in all)
    (dict(T=16383, K=(1 << 21) - 16, top=1, E=8, I=16), dict(T=16384, K=(1 << 21) - 16, top=1, E=8, I=16)),
    (dict(T=(1 << 25) - (1 << 11), K=1 << 10, top=1, E=8, I=16), dict(T=(1 << 25) - (1 << 11) + 1, K=1 << 10, top=1, E=8, I=16)),
    # the activation, where it is a launch of its own
    (dict(T=16 * BLOCKS, K=16, top=1, E=1, I=16), dict(T=16 * BLOCKS + 1, K=16, top=1, E=1, I=16)),
    (dict(T=8 * BLOCKS, K=16, top=2, E=8, I=16), dict(T=8 * BLOCKS + 1, K=16, top=2, E=8, I=16)),
    (dict(T=2 * BLOCKS, K=16, top=4, E=8, I=208), dict(T=2 * BLOCKS + 1, K=16, top=4, E=8, I=208)),
])
def test_sizes_of_the_experts(lib, inside, outside):
    size = lambda s: lib.aq_fp8_experts_workspace(s["T"], s["top"], s["K"], s["E"], s["I"])
    assert size(inside) > 0 == size(outside)
    _limit(_x, lib, dict(inside, wb=BIG), dict(outside, wb=BIG), "too large")


@pytest.mark.parametrize("T,top", [(4, 1 << 62), (1 << 29, 1 << 35), (1 << 20, (1 << 44) + 1), (3, (1 << 63) - 1), (2, 1 << 31)])
def test_choices_whose_product_overflows(lib, T, top):
    """T * top past 64 bits, some of them small again."""
    assert _g(lib, T=T, top=top, W=1 << 16, wb=BIG) == _lib.AQ_EINVAL and "top" in _lib.last_error()
    assert _c(lib, T=T, top=top) == _cb(lib, T=T, top=top) == _r(lib, T=T, top=top) == _b(lib, T=T, top=top) == _lib.AQ_EINVAL
    assert _x(lib, T=T, top=top, wb=BIG) == _lib.AQ_EINVAL and "top" in _lib.last_error()
    assert lib.aq_moe_group_workspace(T, top, 8) == lib.aq_fp8_experts_workspace(T, top, 256, 8, 128) == 0
