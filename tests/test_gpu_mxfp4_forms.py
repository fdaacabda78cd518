"""Every form of the MXFP4 products on random data that a wrong permutation of rows, columns, k or factors would show.

A16: whole numbers to 8 times weights to 6 in steps of 1/4; A4: activations to 6 in steps of 1/4 times weights to 12 in
steps of 1/2.  A sum of K products is a multiple of 1/4 below 48 K, or of 1/8 below 72 K: for K below 14500 it fits 24
bits, every order of additions is exact, and outputs are compared for equality.
"""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as O
from tests.gpu_util import host, step
from tests.mxfp4_forms import SIZES, form_of

pytestmark = pytest.mark.gpu
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _blocks(g, *lead, k, lo):
    """Random codes and factors of 2^lo and 2^(lo + 1)."""
    return (torch.randint(0, 256, (*lead, k // 2), generator=g, device="cuda", dtype=U8),
            torch.randint(127 + lo, 129 + lo, (*lead, k // 32), generator=g, device="cuda", dtype=U8))


def _values(codes, scales):
    """The values of MXFP4 blocks in 64 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return v * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)


def _activations(g, rows, k, a4):
    """(the call's arguments, values): A16 rows lie apart in a matrix that is NaN elsewhere."""
    if a4:
        pair = _blocks(g, rows, k=k, lo=-1)
        return pair, _values(*pair)
    wide = torch.full((rows, k + 40), float("nan"), dtype=BF16, device="cuda")
    x = wide[:, 24:24 + k]
    x.copy_(torch.randint(-8, 9, (rows, k), generator=g, device="cuda"))
    return (x,), x.double()


def _guarded(m, n, dtype):
    whole = torch.full((m * n + 512,), 77.0, dtype=dtype, device="cuda")
    return whole[256:256 + m * n].view(m, n), whole


def _check(call, ref, what):
    """call(out) into a buffer with a border, in both types of output; rows of ref that are infinite are not written."""
    m, n = ref.shape
    left = torch.isinf(ref)
    for dtype in (F32, BF16):
        out, whole = _guarded(m, n, dtype)
        call(out)
        want = torch.where(left, 77.0, ref).to(F32).to(dtype)
        assert torch.equal(torch.nan_to_num(out, nan=-1e30), torch.nan_to_num(want, nan=-1e30)), (what, dtype)
        assert bool((whole[:256] == 77).all()) and bool((whole[256 + m * n:] == 77).all()), (what, dtype)


def test_values_are_the_oracles():
    g = torch.Generator(device="cuda").manual_seed(1)
    c, s = _blocks(g, 7, k=96, lo=-1)
    assert np.array_equal(host(_values(c, s)), O.dequantize(host(c), host(s)))


@pytest.mark.parametrize("a4,grouped,name", [key for key in SIZES if not key[1]])
def test_dense_form(lib, a4, grouped, name):
    from weight_only_bit_group_amd import binding as B
    call = B.aq_mxfp4_gemm_a4 if a4 else B.aq_mxfp4_gemm
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    for m, n, k in SIZES[a4, grouped, name]:
        assert form_of(lib, a4, False, m, n, k, cus=cus) == name
        step(f"mxfp4 gemm {name} a4={a4} {m}x{n}x{k}")
        g = torch.Generator(device="cuda").manual_seed(m + n + k)
        c, s = _blocks(g, n, k=k, lo=0 if a4 else -1)
        x, xv = _activations(g, m, k, a4)
        _check(lambda out: call(*x, c, s, out=out), xv @ _values(c, s).t(), (m, n, k))


@pytest.mark.parametrize("a4,grouped,name", [key for key in SIZES if key[1]])
def test_grouped_form(lib, a4, grouped, name):
    """Ragged experts, some without a row; rows before the first and behind the last; with and without a row list, which
    holds repeated rows and rows outside X."""
    from weight_only_bit_group_amd import binding as B
    call = B.aq_mxfp4_grouped_gemm_a4 if a4 else B.aq_mxfp4_grouped_gemm
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    for i, (m, n, k, e) in enumerate(SIZES[a4, grouped, name]):
        assert form_of(lib, a4, True, m, n, k, e, cus=cus) == name
        step(f"mxfp4 grouped {name} a4={a4} {m}x{n}x{k} of {e}")
        g = torch.Generator(device="cuda").manual_seed(m + n + k)
        c, s = _blocks(g, e, n, k=k, lo=0 if a4 else -1)
        rng = np.random.default_rng(m + n + k)
        first, end = (1, m - 2) if m > 8 else (0, m)
        share = rng.dirichlet(np.where(rng.random(e) < 0.3, 1e-3, 1.0))
        off = first + np.concatenate([[0], np.cumsum(rng.multinomial(end - first, share))])
        gather = i % 3 != 2
        t = m // 2 + 1 if gather else m
        x, xv = _activations(g, t, k, a4)
        src = rng.integers(0, t, m) if gather else np.arange(m)
        rows = src.copy()
        if gather:
            rows[m // 3], rows[m - 1 - m // 4] = -1, t
        lost = rows != src
        # (zeros where the values are not used: rows of no expert are not written, lost ones are NaN)
        ref = torch.full((m, n), float("inf"), dtype=torch.float64, device="cuda")
        at = torch.from_numpy(src).cuda()
        for j in range(e):
            lo, hi = int(off[j]), int(off[j + 1])
            if hi > lo:
                ref[lo:hi] = xv[at[lo:hi]] @ _values(c[j], s[j]).t()
        own = torch.zeros(m, dtype=torch.bool, device="cuda")
        own[first:end] = True
        ref[torch.from_numpy(lost).cuda() & own] = float("nan")
        lists = dict(rows=torch.from_numpy(rows.astype(np.int32)).cuda()) if gather else {}
        offsets = torch.from_numpy(off.astype(np.int32)).cuda()
        _check(lambda out: call(*x, c, s, offsets, out=out, **lists), ref, (m, n, k, e))


@pytest.mark.parametrize("a4,grouped,name", [key for key in SIZES if not key[1]])
def test_what_is_not_finite_stays_in_its_row_and_column(lib, a4, grouped, name):
    """A NaN factor in the last block of a weight row; an infinity at the end of an activation row (A16) or a NaN factor
    in an activation row's first block (A4): that column and that row, nothing else."""
    from weight_only_bit_group_amd import binding as B
    call = B.aq_mxfp4_gemm_a4 if a4 else B.aq_mxfp4_gemm
    for m, n, k in SIZES[a4, grouped, name][1:4]:
        step(f"mxfp4 gemm {name} a4={a4} {m}x{n}x{k}, values that are not finite")
        g = torch.Generator(device="cuda").manual_seed(m + n + k)
        c, s = _blocks(g, n, k=k, lo=0 if a4 else -1)
        c[:, -1] |= 0x22   # no zero weight under the infinity
        x, xv = _activations(g, m, k, a4)
        ref = (xv @ _values(c, s).t()).float()
        row, col = m // 2, n // 3
        s[col, -1] = 255
        if a4:
            x[1][row, 0] = 255
        else:
            x[0][row, -1] = float("inf")
        y = call(*x, c, s)
        rows, cols = torch.arange(m, device="cuda") != row, torch.arange(n, device="cuda") != col
        assert bool(y[:, col].isnan().all())
        assert bool(y[row][cols].isnan().all() if a4 else y[row][cols].isinf().all())
        assert torch.equal(y[rows][:, cols], ref[rows][:, cols])


def _few_codes(g, *lead, k):
    """Codes of 0, 1 and -1 with factors 1: sums of K below 2^24 products are exact."""
    nibbles = torch.tensor([0, 2, 10], dtype=U8, device="cuda")
    pick = torch.randint(0, 3, (2, *lead, k // 2), generator=g, device="cuda")
    return nibbles[pick[0]] | (nibbles[pick[1]] << 4), torch.full((*lead, k // 32), 127, dtype=U8, device="cuda")


@pytest.mark.parametrize("a4", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 19, (1 << 22) - 32), (3, 40, 2097184), (150, 70, 1048608), (2000003, 9, 64), (5, 4194303, 32)])
def test_longest_rows_and_tallest_matrices(a4, m, n, k):
    """Rows of nearly 2^22 k, two million rows, the most columns."""
    from weight_only_bit_group_amd import binding as B
    step(f"mxfp4 gemm a4={a4} {m}x{n}x{k}")
    g = torch.Generator(device="cuda").manual_seed(m + n)
    c, s = _few_codes(g, n, k=k)
    if a4:
        x = _few_codes(g, m, k=k)
        xv = _values(*x)
        y = B.aq_mxfp4_gemm_a4(*x, c, s)
    else:
        xv = torch.randint(-1, 2, (m, k), generator=g, device="cuda").double()
        y = B.aq_mxfp4_gemm(xv.to(BF16), c, s)
    assert torch.equal(y, (xv @ _values(c, s).t()).float())


@pytest.mark.parametrize("a4", [False, True])
@pytest.mark.parametrize("m,e", [(1000, 70001), (5, 1000003)])
def test_very_many_experts(a4, m, e):
    from weight_only_bit_group_amd import binding as B
    n, k = 17, 64
    step(f"mxfp4 grouped a4={a4} {m} rows over {e} experts")
    g = torch.Generator(device="cuda").manual_seed(e)
    c, s = _few_codes(g, e, n, k=k)
    chosen = torch.sort(torch.randint(0, e, (m,), generator=g, device="cuda"))[0]
    chosen[-1] = e - 1
    off = torch.searchsorted(chosen, torch.arange(e + 1, device="cuda"), out_int32=True)
    if a4:
        x = _few_codes(g, m, k=k)
        xv = _values(*x)
        y = B.aq_mxfp4_grouped_gemm_a4(*x, c, s, off)
    else:
        xv = torch.randint(-1, 2, (m, k), generator=g, device="cuda").double()
        y = B.aq_mxfp4_grouped_gemm(xv.to(BF16), c, s, off)
    ref = (xv.unsqueeze(1) * _values(c[chosen], s[chosen])).sum(-1)
    assert torch.equal(y, ref.float())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_and_read_back_beyond_32_bits(dtype):
    """A matrix of more than 2^32 elements: every slice of rows as quantised by itself, and read back."""
    from weight_only_bit_group_amd import binding as B
    m, k = 66000, 65536 + 32
    assert m * k > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(m, k, dtype=dtype, device="cuda").normal_(generator=g)
    step(f"aq_mxfp4_quantize {m}x{k} {dtype}")
    c, s = B.aq_mxfp4_quantize(x)
    y = B.aq_mxfp4_dequantize(c, s, out_dtype=dtype)
    for lo in range(0, m, 6000):
        part = slice(lo, min(lo + 6000, m))
        c1, s1 = B.aq_mxfp4_quantize(x[part])
        assert torch.equal(c[part], c1) and torch.equal(s[part], s1)
        assert torch.equal(y[part], B.aq_mxfp4_dequantize(c1, s1, out_dtype=dtype))
