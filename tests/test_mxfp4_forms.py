"""Every form of the MXFP4 products is compiled for some size that the tests run (no GPU: the choice is the host's)."""
import pytest

from tests.mxfp4_forms import SIZES, form_of, forms


@pytest.mark.parametrize("a4", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_every_form_has_sizes(lib, a4, grouped):
    names = [name for name in forms(lib, a4, grouped) if name]
    assert len(set(names)) == len(names) > 4
    assert set(names) == {name for kind, group, name in SIZES if (kind, group) == (a4, grouped)}


@pytest.mark.parametrize("a4,grouped,name", list(SIZES))
def test_sizes_select_their_form(lib, a4, grouped, name):
    sizes = SIZES[a4, grouped, name]
    assert len(sizes) >= 4
    for size in sizes:
        assert form_of(lib, a4, grouped, *size) == name, size


def test_few_rows_of_many_columns_take_a_tile(lib):
    """The form of one wave over 64 columns is for experts; dense products of MXFP4 activations run faster in tiles."""
    for m, n, k in ((1, 131072, 2048), (16, 200000, 2048), (4, 120000, 256)):
        assert form_of(lib, True, False, m, n, k) == "tile 2 x 2 of 2 x 4"
