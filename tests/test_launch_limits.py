"""The largest sizes that the routing and FP8 entry points accept are the largest that their launches can take (fewer than
2^32 threads); larger ones are refused before anything is launched.  (No GPU: with a failure injected in front of the
launch, a call whose arguments are accepted ends there.)"""
import pytest

from tests.test_moe_abi import _b, _r
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
