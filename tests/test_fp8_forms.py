"""Every form of the FP8 products is compiled for some size that the tests run (no GPU: the choice is the host's)."""
import pytest

from tests.fp8_forms import CUS, GATED, ROUNDED, SIZES, form_of, forms


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
def test_every_form_has_sizes(lib, bf16, grouped):
    names = forms(lib, bf16)
    assert len(set(names)) == len(names) > 4
    assert set(names) == {name for kind, group, name in SIZES if (kind, group) == (bf16, grouped)}


@pytest.mark.parametrize("bf16,grouped,name", list(SIZES))
def test_sizes_select_their_form(lib, bf16, grouped, name):
    sizes = SIZES[bf16, grouped, name]
    assert len(sizes) >= 2
    for size in sizes:
        assert form_of(lib, bf16, *size) == name, size


def test_gated_sizes_select_their_form(lib):
    assert set(GATED) == {-1, 0, 1}
    for form, sizes in GATED.items():
        assert len(sizes) >= 2
        for t, top, e, k, inner in sizes:
            assert lib.fp8_gated_form(t * top, k, inner, e, CUS) == form, (t, top, e, k, inner)


def test_gated_activation_alone_where_it_has_to_be(lib):
    """A last block of h that is not whole, and an expert's weights past 32 bits of offset."""
    assert lib.fp8_gated_form(16384, 2048, 1408, 64, CUS) >= 0 > lib.fp8_gated_form(16384, 2048, 1424, 64, CUS)
    assert all(lib.fp8_gated_form(1 << i, 1 << 15, 1 << 16, 2, CUS) < 0 for i in range(20))


def test_rounded_sizes_select_their_form(lib):
    assert {name for _, name in ROUNDED} == {name for name in forms(lib, True) if name.startswith("split 1 ")}
    for (bf16, name), sizes in ROUNDED.items():
        assert len(sizes) >= 3 and all(m <= 16 and m * k <= 8192 and form_of(lib, bf16, m, n, k) == name for m, n, k in sizes)
