"""Every form of the FP8 products on random data that a wrong permutation of rows, columns, k or scales would show.

Whole numbers of -8 .. 8 times whole numbers of -8 .. 8, scales of 1/2, 1 and 2: products lie within 2^13 of each other
and a sum of K of them is a multiple of 1/4 below 256 K, which for K below 16384 fits 24 bits, so every order of
additions is exact.  Outputs are compared for equality, in bf16 after the one rounding.
"""
import pytest
import torch

from tests.fp8_forms import SIZES, form_of
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrix(g, *shape, rows):
    """(codes, scales, 64-bit values) of a matrix or a stack of them."""
    v = torch.randint(-8, 9, shape, generator=g, device="cuda").float()
    s = torch.exp2(torch.randint(-1, 2, (*shape[:-2], -(-shape[-2] // rows), -(-shape[-1] // 128)), generator=g, device="cuda").float())
    full = s.double().repeat_interleave(rows, -2)[..., :shape[-2], :].repeat_interleave(128, -1)[..., :shape[-1]]
    return v.to(F8), s, v.double() * full


def _guarded(m, n, dtype):
    whole = torch.full((m * n + 512,), 77.0, dtype=dtype, device="cuda")
    return whole[256:256 + m * n].view(m, n), whole


@pytest.mark.parametrize("bf16,grouped,name", list(SIZES))
def test_form(lib, bf16, grouped, name):
    from weight_only_bit_group_amd import binding as B
    dtype = BF16 if bf16 else F32
    for size in SIZES[bf16, grouped, name]:
        assert torch.cuda.get_device_properties(0).multi_processor_count != 256 or form_of(lib, bf16, *size) == name
        m, n, k = size[:3]
        step(f"fp8 {name} {'bf16' if bf16 else 'fp32'} {size}")
        g = torch.Generator(device="cuda").manual_seed(m * n + k)
        out, whole = _guarded(m, n, dtype)
        if not grouped:
            xc, xs, xv = _matrix(g, m, k, rows=1)
            wc, ws, wv = _matrix(g, n, k, rows=128)
            B.aq_fp8_gemm(xc, xs, wc, ws, out=out)
            ref = xv @ wv.t()
        else:
            e, t = size[3], max(1, m // 3)
            xc, xs, xv = _matrix(g, t, k, rows=1)
            wc, ws, wv = _matrix(g, e, n, k, rows=128)
            cuts = torch.randint(0, m + 1, (e - 1,), generator=g, device="cuda").sort()[0]
            off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), m)]).int()
            off[0] = min(1, int(off[1]))                       # (a row in front of the first expert: not written)
            rows = torch.randint(0, t, (m,), generator=g, device="cuda").int()
            rows[m // 2] = t                                   # (outside X)
            B.aq_fp8_grouped_gemm(xc, xs, wc, ws, off, rows, out=out)
            ref = torch.full((m, n), 77.0, dtype=torch.float64, device="cuda")
            lo = off.tolist()
            for i in range(e):
                if lo[i + 1] > lo[i]:
                    ref[lo[i]:lo[i + 1]] = xv[rows[lo[i]:lo[i + 1]].long().clamp(max=t - 1)] @ wv[i].t()
            lost = (rows == t) & (torch.arange(m, device="cuda") >= lo[0])
            assert out[lost].isnan().all()
            ref[lost] = 0
            out[lost] = 0
        assert torch.equal(out, ref.to(dtype)), size
        assert (whole[:256] == 77).all() and (whole[256 + m * n:] == 77).all()


@pytest.mark.parametrize("bf16,grouped,name", [k for k in SIZES if not k[1]])
def test_row_and_column_edges(lib, bf16, grouped, name):
    """One row or column more and less than whole tiles of every form."""
    from weight_only_bit_group_amd import binding as B
    m, n, k = SIZES[bf16, grouped, name][0]
    step(f"fp8 {name} edges of {m} x {n} x {k}")
    g = torch.Generator(device="cuda").manual_seed(1)
    xc, xs, xv = _matrix(g, m + 1, k, rows=1)
    wc, ws, wv = _matrix(g, n + 1, k, rows=128)
    ref = (xv @ wv.t()).to(BF16 if bf16 else F32)
    for r in (max(1, m - 1), m, m + 1):
        for c in (max(1, n - 1), n, n + 1):
            nb = -(-c // 128)
            out, whole = _guarded(r, c, ref.dtype)
            B.aq_fp8_gemm(xc[:r], xs[:r], wc[:c], ws[:nb], out=out)
            assert torch.equal(out, ref[:r, :c]), (r, c)
            assert (whole[:256] == 77).all() and (whole[256 + r * c:] == 77).all()
