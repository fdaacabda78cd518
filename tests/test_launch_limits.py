"""The largest sizes that the routing and FP8 entry points accept are the largest that their launches can take (fewer than
2^32 threads); larger ones are refused before anything is launched.  (No GPU: with a failure injected in front of the
launch, a call whose arguments are accepted ends there.)"""
import pytest

from tests.test_moe_abi import _b, _c, _cb, _r
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
