"""The experts' call in all of its forms, bit for bit against the calls that it is made of.

x holds whole numbers of -7 .. 7 with a 7 in every block of 128, so its codes are exact with scales of 1 / 64; the
weights of the first product are such numbers times powers of two, and every order of additions is exact: g and u have
the same bits in every form, and with them the codes of h.  The second product's weights pick one column of h times a power
of two for every output, one product each, exact on both kinds of matrix instructions.
"""
import pytest
import torch

from tests.fp8_forms import GATED
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(t, top, e, k, inner, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + t + k)

    def whole(*shape):
        return torch.randint(-7, 8, shape, generator=g, device="cuda").float()

    def power(lo, hi, *shape):
        return torch.exp2(torch.randint(lo, hi + 1, shape, generator=g, device="cuda").float())

    x = whole(t, k)
    x[:, ::128] = 7
    gu = whole(e, 2 * inner, k).to(F8), power(-11, -9, e, -(-2 * inner // 128), -(-k // 128))
    pick = torch.randint(0, inner, (e, k, 1), generator=g, device="cuda")
    down = torch.zeros(e, k, inner, device="cuda").scatter_(2, pick, power(-2, 2, e, k, 1)).to(F8), power(-1, 1, e, -(-k // 128), -(-inner // 128))
    ids = torch.randint(-1, e + 1, (t, top), generator=g, device="cuda").int()
    weights = torch.rand(t, top, generator=g, device="cuda")
    return x.to(BF16), gu, down, ids, weights


def _apart(x, gu, down, ids, weights, out):
    from weight_only_bit_group_amd import binding as B
    offsets, rows, slots = B.aq_moe_group(ids, gu[0].shape[0])
    codes, scales = B.aq_fp8_quantize(x)
    assert (scales == 1 / 64).all()
    h = B.aq_fp8_swiglu_quantize(B.aq_fp8_grouped_gemm(codes, scales, *gu, offsets, rows), offsets[-1:])
    y = B.aq_fp8_grouped_gemm(*h, *down, offsets)
    return B.aq_moe_combine(y, slots, weights, out), y, slots


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("form", list(GATED))
def test_forms(lib, form, out):
    from weight_only_bit_group_amd import binding as B
    for t, top, e, k, inner in GATED[form]:
        step(f"experts {out} form {form}: t {t} top {top} e {e} k {k} inner {inner}")
        args = _inputs(t, top, e, k, inner)
        ref, ry, rslots = _apart(*args, out)
        x, gu, down, ids, weights = args
        got, y, slots = B.aq_fp8_experts(x, *gu, *down, ids, weights, out)
        assert torch.equal(slots, rslots) and got.dtype == out and y.dtype == F32
        used = slots[slots >= 0].long()
        assert torch.equal(y[used], ry[used]), (t, top, e, k, inner)
        assert torch.equal(got, ref), (t, top, e, k, inner)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("inner", [128, 144, 1408])
def test_fills_nothing_else(out, inner):
    """The workspace and the products behind the last expert's rows, and what lies around every output, stay as they were."""
    from weight_only_bit_group_amd import _lib, binding as B
    t, top, e, k = 37, 3, 5, 272
    x, gu, down, ids, weights = _inputs(t, top, e, k, inner)
    ids[5:9] = -1
    need = B.aq_fp8_experts_workspace(t, top, k, e, inner)
    work = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    step(f"experts {out} with guards, inner {inner}")
    got, y, slots = B.aq_fp8_experts(x, *gu, *down, ids, weights, out, workspace=work[256:256 + need])
    assert (work[:256] == 77).all() and (work[256 + need:] == 77).all()
    ref = _apart(x, gu, down, ids, weights, out)[0]
    assert torch.equal(got, ref) and (got[5:9] == 0).all()
    products = torch.full((t * top + 2, k), 77.0, device="cuda")
    small = torch.full((t + 2, k), 77.0, device="cuda", dtype=out)
    where = torch.full(((t + 2) * top,), 77, device="cuda", dtype=torch.int32)
    st = _lib.load().aq_fp8_experts(x.data_ptr(), 1, t, k, k, gu[0].data_ptr(), gu[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), e,
                                    inner, ids.data_ptr(), weights.data_ptr(), top, products[1:].data_ptr(), where[top:].data_ptr(),
                                    small[1:].data_ptr(), 0 if out == F32 else 1, work[256:].data_ptr(), need,
                                    torch.cuda.current_stream().cuda_stream)
    assert st == _lib.AQ_OK
    used = int((slots >= 0).sum())
    assert torch.equal(small[1:-1], ref) and (small[0] == 77).all() and (small[-1] == 77).all()
    assert (products[0] == 77).all() and (products[1 + used:] == 77).all() and torch.equal(products[1:1 + used], y[:used])
    assert (where[:top] == 77).all() and (where[-top:] == 77).all() and torch.equal(where[top:-top].view(t, top), slots)


@pytest.mark.parametrize("out", [F32, BF16])
def test_values_that_are_not_finite(out):
    """A NaN or infinity in a token's block makes that token's output NaN and no other's."""
    from weight_only_bit_group_amd import binding as B
    t, top, e, k, inner = 600, 2, 3, 256, 384
    x, gu, down, ids, weights = _inputs(t, top, e, k, inner)
    ids = ids.clamp(0, e - 1)
    step(f"experts {out} with NaN and infinities")
    clean = B.aq_fp8_experts(x, *gu, *down, ids, weights, out)[0]
    x[7, 3], x[300, 200], x[301, 0] = float("nan"), float("inf"), -float("inf")
    got = B.aq_fp8_experts(x, *gu, *down, ids, weights, out)[0]
    bad = torch.zeros(t, dtype=torch.bool, device="cuda")
    bad[[7, 300, 301]] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])


def test_large_activations_overflow_to_nan_alone():
    """g u past the largest fp32 number is an infinity: its block of h, and the outputs that read it, become NaN."""
    from weight_only_bit_group_amd import binding as B
    t, top, e, k, inner = 700, 1, 2, 128, 128
    x, gu, down, ids, weights = _inputs(t, top, e, k, inner)
    ids.clamp_(0, e - 1)
    up = gu[1].clone()
    up[:] = 2.0 ** 60
    step("experts, overflow of the gated activation")
    args = x, (gu[0], up), down, ids, weights
    assert B.aq_fp8_experts(*args[:1], *args[1], *down, ids, weights, F32)[0].isnan().any(1).all()
    ref = _apart(*args, F32)[0]
    assert torch.equal(torch.nan_to_num(B.aq_fp8_experts(x, *args[1], *down, ids, weights, F32)[0], 5.0), torch.nan_to_num(ref, 5.0))


@pytest.mark.parametrize("t,top,e", [(1, 1, 1), (3, 7, 1024), (40, 6, 600), (1024, 16, 700), (2048, 8, 300), (2049, 8, 5), (5000, 4, 1024)])
def test_grouping_beside_the_rounding(t, top, e):
    """Choices of one expert to 1024, with one workgroup (up to 16384 choices) and with three kernels behind it; fp32 rows apart."""
    from weight_only_bit_group_amd import binding as B
    k, inner = 144, 32
    x, gu, down, ids, weights = _inputs(t, top, e, k, inner)
    step(f"experts: {t} tokens of {top} choices of {e}")
    ref, _, rslots = _apart(x, gu, down, ids, weights, F32)
    wide = torch.full((t, k + 20), float("nan"), device="cuda")
    wide[:, :k] = x.float()
    for rows in (x, wide[:, :k]):
        got, _, slots = B.aq_fp8_experts(rows, *gu, *down, ids, weights, F32)
        assert torch.equal(slots, rslots) and torch.equal(got, ref)
