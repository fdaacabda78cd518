"""Few short rows, rounded to FP8 by the product itself: the bits of the rounding and the product as two calls."""
import pytest
import torch

from tests.fp8_forms import ROUNDED
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _two_calls(x, codes, scales, out):
    from weight_only_bit_group_amd import binding as B
    return B.aq_fp8_gemm(*B.aq_fp8_quantize(x), codes, scales, out_dtype=out)


def _bits(t):
    return torch.nan_to_num(t.float(), nan=5e4, posinf=6e4, neginf=-6e4)   # (a NaN's payload is not part of it)


@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("bf16,name", list(ROUNDED))
def test_rounded_by_the_product(lib, bf16, name, x_dtype):
    from weight_only_bit_group_amd import binding as B
    out = BF16 if bf16 else F32
    for m, n, k in ROUNDED[bf16, name]:
        step(f"fp8 linear {name}, {x_dtype} rows {m} x {n} x {k} to {out}")
        g = torch.Generator(device="cuda").manual_seed(m + n + k)
        codes, scales = B.aq_fp8_quantize(torch.randn(n, k, generator=g, device="cuda"), 128)
        ld = k + 24 if x_dtype == F32 else k + 40
        held = torch.full((m + 2, ld), float("nan"), dtype=x_dtype, device="cuda")   # rows apart, among values never read
        x = held[1:-1, :k]
        x.copy_(torch.randn(m, k, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 30, (m, k), generator=g, device="cuda").float()))
        whole = torch.full((m * n + 512,), 77.0, dtype=out, device="cuda")
        y = whole[256:256 + m * n].view(m, n)
        assert B.aq_fp8_linear(x, codes, scales, out=y) is y
        ref = _two_calls(x.contiguous(), codes, scales, out)
        assert torch.equal(y, ref), (m, n, k)
        assert (whole[:256] == 77).all() and (whole[256 + m * n:] == 77).all()
        assert torch.equal(B.aq_fp8_linear(x.contiguous(), codes, scales, out), ref)


def test_values_at_the_ends(lib):
    """Zeros, the least and largest numbers, NaN and infinities: as the two calls, and no row's reach another's."""
    from weight_only_bit_group_amd import binding as B
    codes, scales = B.aq_fp8_quantize(torch.randn(500, 272, device="cuda"), 128)
    x = torch.randn(8, 272, device="cuda")
    x[0] = 0
    x[1] = -0.0
    x[2] = 1e-45
    x[3, 5], x[4, 200], x[5, 271] = float("nan"), float("inf"), -float("inf")
    x[6] = 3e38
    x[7, 0] = 1e-30
    step("fp8 linear, values at the ends")
    for v in (x, x.to(BF16)):
        for out in (F32, BF16):
            y = B.aq_fp8_linear(v, codes, scales, out)
            assert torch.equal(_bits(y), _bits(_two_calls(v, codes, scales, out)))
            assert y[3:6].isnan().all() and not y[:3].isnan().any() and not y[7].isnan().any()


def test_at_the_limit(lib):
    """8192 values and 8208, 16 rows and 17: with the rounding inside and in front, the same as two calls."""
    from weight_only_bit_group_amd import binding as B
    for m, n, k in ((1, 300, 8192), (1, 300, 8208), (16, 300, 512), (16, 300, 528), (17, 300, 464), (2, 70, 4096), (4, 70, 2048), (16, 4, 16)):
        step(f"fp8 linear {m} x {n} x {k}")
        codes, scales = B.aq_fp8_quantize(torch.randn(n, k, device="cuda"), 128)
        x = torch.randn(m, k, device="cuda")
        for out in (F32, BF16):
            assert torch.equal(B.aq_fp8_linear(x, codes, scales, out), _two_calls(x, codes, scales, out))


def test_captured_and_on_two_streams(lib):
    from weight_only_bit_group_amd import binding as B
    codes, scales = B.aq_fp8_quantize(torch.randn(3000, 1024, device="cuda"), 128)
    xs = [torch.randn(m, 1024, device="cuda").to(BF16) for m in (1, 6)]
    step("fp8 linear of few rows, captured, and on two streams")
    refs = [_two_calls(x, codes, scales, F32) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(B.aq_fp8_linear(x, codes, scales))
    torch.cuda.synchronize()
    assert all(torch.equal(y, refs[i % 2]) for i, y in enumerate(got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = B.aq_fp8_linear(xs[1], codes, scales)
    for _ in range(3):
        xs[1].normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, _two_calls(xs[1], codes, scales, F32))
