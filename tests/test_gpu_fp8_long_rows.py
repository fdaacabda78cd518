"""FP8 products whose waves take more than 64 stages of k: the weights' scales are held 64 stages at a time.

Whole numbers of -2 .. 2 times whole numbers of -2 .. 2, scales of 1/2, 1 and 2 drawn for every block: a sum of K products
is a multiple of 1/4 below 16 K, which for K below 2^18 fits 24 bits, so every order of additions is exact and outputs are
compared for equality.
"""
import pytest
import torch

from tests.fp8_forms import SIZES, form_of
from tests.gpu_util import step
from tests.test_gpu_fp8_forms import _guarded

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn

# (bf16 out, grouped, form): one stage, or a few, past 64 of a wave; past 128.  (16 x 16 over 4 waves is taken for fewer
# stages only.)
LONG = {
    (True, False, "split 1 x 1 over 16"): [(1, 1, 131088)],
    (True, False, "split 1 x 2 over 8"): [(537, 146, 65552), (645, 143, 132112)],
    (True, False, "split 1 x 4 over 8"): [(257, 298, 65552), (338, 228, 131200)],
    (True, False, "split 2 x 2 over 8"): [(540, 589, 65584), (668, 458, 131200)],
    (True, False, "split 2 x 4 over 4"): [(878, 676, 32912), (771, 810, 66064)],
    (True, True, "split 1 x 1 over 16"): [(1, 1, 131088, 3)],
    (True, True, "split 1 x 2 over 8"): [(497, 148, 66576, 7), (636, 132, 131216, 7)],
    (True, True, "split 1 x 4 over 8"): [(210, 294, 65584, 7), (213, 305, 131088, 7)],
    (True, True, "split 2 x 2 over 8"): [(669, 454, 65680, 2), (639, 516, 131088, 2)],
    (True, True, "split 2 x 4 over 4"): [(712, 743, 32784, 7), (703, 804, 65584, 7)],
    (False, False, "split 1 x 1 over 16"): [(1, 1, 131088)],
    (False, False, "split 1 x 2 over 8"): [(354, 350, 65584)],
    (False, False, "split 1 x 4 over 8"): [(1, 13622, 65584), (3, 13880, 131216)],
    (False, False, "split 2 x 2 over 8"): [(378, 404, 65664), (338, 470, 131216)],
    (False, False, "split 2 x 4 over 4"): [(961, 826, 32816), (810, 1005, 65664)],
    (False, True, "split 1 x 1 over 16"): [(1, 1, 131088, 3)],
    (False, True, "split 1 x 2 over 8"): [(254, 405, 65584, 7)],
    (False, True, "split 1 x 4 over 8"): [(90, 1520, 65680, 7), (95, 1468, 131088, 7)],
    (False, True, "split 2 x 2 over 8"): [(423, 350, 65552, 7), (355, 420, 131120, 7)],
    (False, True, "split 2 x 4 over 4"): [(789, 865, 32816, 7), (822, 888, 65552, 7)],
}


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrix(g, *shape, rows):
    v = torch.randint(-2, 3, shape, generator=g, device="cuda").float()
    s = torch.exp2(torch.randint(-1, 2, (*shape[:-2], -(-shape[-2] // rows), -(-shape[-1] // 128)), generator=g, device="cuda").float())
    full = s.repeat_interleave(rows, -2)[..., :shape[-2], :].repeat_interleave(128, -1)[..., :shape[-1]]
    return v.to(F8), s, v * full


def _exact(x, w):
    """x w^T in 64 bits, some k at a time."""
    return sum(a.double() @ b.double().t() for a, b in zip(x.split(1 << 14, 1), w.split(1 << 14, 1)))


@pytest.mark.parametrize("bf16,grouped,name", list(LONG))
def test_more_than_64_stages_of_a_wave(lib, bf16, grouped, name):
    from weight_only_bit_group_amd import binding as B
    dtype = BF16 if bf16 else F32
    for size in LONG[bf16, grouped, name]:
        m, n, k = size[:3]
        assert torch.cuda.get_device_properties(0).multi_processor_count != 256 or form_of(lib, bf16, *size) == name
        assert -(-k // 128) > 64 * int(name.split()[-1]) and (bf16, grouped, name) in SIZES
        step(f"fp8 {name} {'bf16' if bf16 else 'fp32'} {size}")
        g = torch.Generator(device="cuda").manual_seed(k)
        out, whole = _guarded(m, n, dtype)
        xc, xs, xv = _matrix(g, m, k, rows=1)
        if not grouped:
            wc, ws, wv = _matrix(g, n, k, rows=128)
            B.aq_fp8_gemm(xc, xs, wc, ws, out=out)
            ref = _exact(xv, wv)
        else:
            e = size[3]
            wc, ws, wv = _matrix(g, e, n, k, rows=128)
            cuts = torch.randint(0, m + 1, (e - 1,), generator=g, device="cuda").sort()[0]
            off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), m)]).int()
            B.aq_fp8_grouped_gemm(xc, xs, wc, ws, off, None, out=out)
            lo = off.tolist()
            ref = torch.cat([_exact(xv[lo[i]:lo[i + 1]], wv[i]) for i in range(e)])
        assert torch.equal(out, ref.to(dtype)), size
        assert (whole[:256] == 77).all() and (whole[256 + m * n:] == 77).all()
