"""The largest sizes that the routing and FP8 entry points accept, launched: rows that repeat a few patterns, compared with
the same rows in a small call."""
import pytest
import torch

from tests.gpu_util import step

pytestmark = pytest.mark.gpu
BLOCKS = (1 << 24) - 1   # workgroups of 256 threads in a launch
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def B():
    from weight_only_bit_group_amd import binding
    return binding


PERIOD = 97


def _rows(few, n):
    """n rows that repeat the PERIOD rows of `few`."""
    whole = n // PERIOD * PERIOD
    return torch.cat([few.expand(n // PERIOD, *few.shape).reshape(whole, *few.shape[1:]), few[:n - whole]])


def _repeats(got, few):
    n = got.shape[0] // PERIOD
    return bool((got[:n * PERIOD].view(n, PERIOD, *few.shape[1:]) == few).all()) and torch.equal(got[n * PERIOD:], few[:got.shape[0] - n * PERIOD])


def test_most_tokens_of_route_and_its_gradient():
    t, how = 4 * BLOCKS, dict(score="sigmoid", scale=1.5)
    few, d = torch.randn(PERIOD, 4, device="cuda").to(BF16), torch.randn(PERIOD, 1, device="cuda")
    ref = B().aq_moe_route(few, 1, **how)
    l = _rows(few, t)
    step(f"route {t} tokens")
    ids, w = B().aq_moe_route(l, 1, **how)
    assert ids.shape == (t, 1) and _repeats(ids, ref[0]) and _repeats(w, ref[1])
    step(f"route's gradient, {t} tokens")
    got = B().aq_moe_route_backward(l, ids, w, _rows(d, t), score="sigmoid", renormalize=False, scale=1.5)
    assert _repeats(got, B().aq_moe_route_backward(few, *ref, d, score="sigmoid", renormalize=False, scale=1.5))
    assert (got != 0).any()
    with pytest.raises(ValueError, match="T must be"):
        B().aq_moe_route(_rows(few, t + 1)[:, :1], 1)


def test_most_choices_of_the_weighted_sums_gradient():
    t, top, r = 2 * BLOCKS, 2, 50
    y, d = torch.randn(r, 8, device="cuda"), torch.randn(PERIOD, 8, device="cuda").to(BF16)
    slots = torch.randint(-1, r + 1, (PERIOD, top), dtype=torch.int32, device="cuda")
    step(f"combine's gradient, {t * top} choices")
    got = B().aq_moe_combine_backward(y, _rows(slots, t), _rows(d, t))
    assert got.shape == (t, top) and _repeats(got, B().aq_moe_combine_backward(y, slots, d)) and (got != 0).any()
    step(f"combine, {t * top} choices")
    w = torch.rand(PERIOD, top, device="cuda")
    got = B().aq_moe_combine(y, _rows(slots, t), _rows(w, t), BF16)
    assert _repeats(got, B().aq_moe_combine(y, slots, w, BF16))
    with pytest.raises(ValueError, match="T \\* top"):
        B().aq_moe_combine_backward(y, _rows(slots, t + 1), _rows(d, t + 1))


def test_most_columns_of_combine():
    """Rows as long as they may be, as many as a launch takes: 64 GiB of bf16, every row one of four."""
    k = (1 << 22) - 8
    t = 2048 * BLOCKS // k
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("not enough memory")
    y = torch.randn(4, k, device="cuda").to(BF16)
    slots = (torch.arange(t, device="cuda", dtype=torch.int32) % 4)[:, None].contiguous()
    step(f"combine {t} x {k}")
    out = B().aq_moe_combine(y, slots, torch.ones(t, 1, device="cuda"), BF16)
    for i in range(4):
        assert all(torch.equal(row, y[i]) for row in out[i::4][::97]) and torch.equal(out[t - 4 + i], y[(t - 4 + i) % 4])
    assert torch.equal(out[:, 0], y[:, 0][slots[:, 0].long()]) and torch.equal(out[:, -1], y[:, -1][slots[:, 0].long()])
    del out
    torch.cuda.empty_cache()


def test_most_blocks_of_the_quantiser():
    few = torch.randn(PERIOD, 1, 16, device="cuda").to(BF16)
    step(f"quantise {BLOCKS} matrices")
    codes, scales = B().aq_fp8_quantize(_rows(few, BLOCKS), 128)
    ref = B().aq_fp8_quantize(few, 128)
    assert scales.shape == (BLOCKS, 1, 1) and _repeats(codes.view(torch.uint8), ref[0].view(torch.uint8)) and _repeats(scales, ref[1])
    with pytest.raises(ValueError, match="128 x 128"):
        B().aq_fp8_quantize(_rows(few, BLOCKS + 1), 128)


def test_most_blocks_of_the_gated_activation():
    m = 16 * BLOCKS
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory")
    few = torch.randn(PERIOD, 32, device="cuda").to(BF16)
    step(f"swiglu quantize {m} rows")
    codes, scales = B().aq_fp8_swiglu_quantize(_rows(few, m))
    ref = B().aq_fp8_swiglu_quantize(few)
    assert codes.shape == (m, 16) and _repeats(codes.view(torch.uint8), ref[0].view(torch.uint8)) and _repeats(scales, ref[1])


def test_most_rows_of_the_quantiser_and_back():
    """2^30 - 64 rows of one block: 32 GiB in, 16 GiB of codes and 4 of scales, 32 GiB back."""
    n = 64 * BLOCKS
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("not enough memory")
    few = torch.randn(128, 16, device="cuda").to(BF16)
    x = few.expand(n // 128, 128, 16).reshape(-1, 16)
    x = torch.cat([x, few[:n - x.shape[0]]]) if n % 128 else x
    ref = B().aq_fp8_quantize(few)
    step(f"quantise {n} rows")
    codes, scales = B().aq_fp8_quantize(x)
    del x

    def repeats(got, ref):
        whole = got.shape[0] // 128
        return all(bool((part == ref).all()) for part in got[:whole * 128].view(whole, 128, *ref.shape[1:]).split(1 << 18)) \
            and torch.equal(got[whole * 128:], ref[:got.shape[0] - whole * 128])

    assert repeats(scales, ref[1]) and repeats(codes.view(torch.uint8), ref[0].view(torch.uint8))
    step(f"read {n} rows back")
    y = B().aq_fp8_dequantize(codes, scales, out_dtype=BF16)
    assert repeats(y, B().aq_fp8_dequantize(*ref, out_dtype=BF16))
    del y, codes, scales
    torch.cuda.empty_cache()
