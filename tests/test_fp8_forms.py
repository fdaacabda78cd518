"""Every form of the FP8 products is compiled for some size that the tests run (no GPU: the choice is the host's)."""
import pytest

from tests.fp8_forms import SIZES, form_of, forms


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_every_form_has_sizes(lib, bf16, grouped):
    names = forms(lib, bf16)
    assert len(set(names)) == len(names) > 4
    assert set(names) == {name for kind, group, name in SIZES if (kind, group) == (bf16, grouped)}


@pytest.mark.parametrize("bf16,grouped,name", list(SIZES))
def test_sizes_select_their_form(lib, bf16, grouped, name):
    sizes = SIZES[bf16, grouped, name]
    assert len(sizes) >= 3
    for size in sizes:
        assert form_of(lib, bf16, *size) == name, size
