"""Every form of the MXFP4 products is compiled for some size that the tests run (no GPU: the choice is the host's)."""
import pytest

from tests.mxfp4_forms import SIZES, form_of, forms


@pytest.mark.parametrize("a4", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_every_form_has_sizes(lib, a4, grouped):
    names = forms(lib, a4, grouped)
    assert len(set(names)) == len(names) > 4
    assert set(names) == {name for kind, group, name in SIZES if (kind, group) == (a4, grouped)}


@pytest.mark.parametrize("a4,grouped,name", list(SIZES))
def test_sizes_select_their_form(lib, a4, grouped, name):
    sizes = SIZES[a4, grouped, name]
    assert len(sizes) >= 4
    for size in sizes:
        assert form_of(lib, a4, grouped, *size) == name, size
