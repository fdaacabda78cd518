"""FP8 quantising and reading back on the GPU against the oracle: every step is a rounding that the definition
names, so codes, scales and values are compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import fp8 as O
from tests.gpu_util import dev, host, step

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def B():
    from weight_only_bit_group_amd import binding
    return binding


def _bytes(codes):
    return host(codes.view(torch.uint8))


def _same(got, ref, what):
    codes, scales = got
    assert codes.dtype == torch.float8_e4m3fn and scales.dtype == F32
    c, s = _bytes(codes), host(scales)
    assert (np.isnan(s) == np.isnan(ref[1])).all() and (np.nan_to_num(s) == np.nan_to_num(ref[1])).all(), what
    assert (c == ref[0]).all(), (what, np.argwhere(c != ref[0])[:5], c[c != ref[0]][:5], ref[0][c != ref[0]][:5])


def _input(rng, *shape):
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal((*shape[:-1], 1)) * 4)
    return x.astype(np.float32)


SIZES = [(1, 16), (1, 128), (3, 48), (16, 2048), (7, 144), (128, 128), (129, 256), (130, 2064), (257, 112), (1, 14336),
         (1000, 16)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,k", SIZES)
def test_quantize_and_read_back(m, k, block_rows, dtype):
    x = dev(_input(np.random.default_rng(m + k), m, k)).to(dtype)
    step(f"fp8 quantize {m} x {k} {dtype} block_rows {block_rows}")
    pair = B().aq_fp8_quantize(x, block_rows)
    _same(pair, O.quantize(host(x.float()), block_rows), "quantize")
    values = O.dequantize(_bytes(pair[0]), host(pair[1])).astype(np.float32)   # one rounding of code times scale
    for out in (F32, BF16):
        y = B().aq_fp8_dequantize(*pair, block_rows, out_dtype=out)
        assert y.dtype == out and (host(y.float()) == host(torch.from_numpy(values).to(out).float())).all()
    y = torch.empty_like(y)
    assert B().aq_fp8_dequantize(pair[0].view(torch.uint8), pair[1], block_rows, out=y) is y


@pytest.mark.parametrize("m,k", [(4100, 2048), (2100, 4080), (20000, 272)])
def test_many_blocks(m, k):
    """Sizes that take several blocks a thread; the last ones end inside a thread's share."""
    x = dev(_input(np.random.default_rng(5), m, k)).to(BF16)
    step(f"fp8 quantize {m} x {k}, many blocks")
    pair = B().aq_fp8_quantize(x)
    rows = np.r_[0:40, m // 2:m // 2 + 40, m - 40:m]
    c, s = O.quantize(host(x.float())[rows])
    assert (_bytes(pair[0])[rows] == c).all() and (host(pair[1])[rows] == s).all()
    y = host(B().aq_fp8_dequantize(*pair))
    assert (y[rows] == O.dequantize(c, s).astype(np.float32)).all()
    # all of it against slices of 40 rows, which take one block a thread
    for lo in range(0, m, 40):
        part = B().aq_fp8_quantize(x[lo:lo + 40])
        assert torch.equal(part[0].view(torch.uint8), pair[0][lo:lo + 40].view(torch.uint8)) and torch.equal(part[1], pair[1][lo:lo + 40])


def test_every_bf16_value_under_many_scales():
    """All finite bf16 values in blocks whose largest value sets scales over the whole range of exponents."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    v = (bits.astype(np.uint32) << 16).view(np.float32)
    v = v[np.isfinite(v)]
    step("fp8 quantize every bf16 value")
    for seed, exps in enumerate((range(-133, -80, 4), range(-80, 128, 12))):
        rng = np.random.default_rng(seed)
        for e in exps:
            top = np.float32(2.0 ** e) * np.float32(1 + rng.integers(0, 128) / 128)
            mine = v[np.abs(v) <= top]
            x = np.zeros((-(-len(mine) // 127), 128), np.float32)
            x[:, 0] = top
            x[:, 1:].reshape(-1)[:0] = 0
            flat = np.zeros(x.shape[0] * 127, np.float32)
            flat[:len(mine)] = mine
            x[:, 1:] = flat.reshape(-1, 127)
            for dtype in (F32, BF16):
                _same(B().aq_fp8_quantize(dev(x).to(dtype)), O.quantize(host(dev(x).to(dtype).float())), f"2^{e}")


def test_borders_between_codes():
    """fp32 values at and next to every middle between two codes, under scales of random mantissas: the quotient's
    rounding decides."""
    rng = np.random.default_rng(7)
    step("fp8 quantize borders")
    rows = []
    for _ in range(300):
        top = np.float32(448) * np.float32(rng.uniform(1, 2)) * np.float32(2.0) ** rng.integers(-100, 100)
        s = top / np.float32(448)
        mids = rng.choice(O._MIDS, 42) * np.float64(s)
        m = mids.astype(np.float32)
        rows.append(np.concatenate([[top, -top], m, np.nextafter(m, np.float32(0)), -np.nextafter(m, np.float32(np.inf))]))
    x = np.array(rows, np.float32)
    _same(B().aq_fp8_quantize(dev(x)), O.quantize(x), "borders")


@pytest.mark.parametrize("block_rows", [1, 128])
def test_special_values(block_rows):
    x = np.random.default_rng(3).standard_normal((260, 272)).astype(np.float32)
    x[0, :] = 0
    x[1, :128] = 1e-42
    x[2, 5] = np.inf
    x[140, 130] = np.nan
    x[141, 271] = -np.inf
    x[150, :] = -0.0
    x[255:, 256:] = 3.4e38
    step(f"fp8 quantize special values, block_rows {block_rows}")
    pair = B().aq_fp8_quantize(dev(x), block_rows)
    _same(pair, O.quantize(x, block_rows), "special")
    y = host(B().aq_fp8_dequantize(*pair, block_rows))
    ref = O.dequantize(*O.quantize(x, block_rows))
    assert (np.isnan(y) == np.isnan(ref)).all() and np.isnan(ref).any()


def test_codes_of_every_byte_are_read_back():
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, 128)
    step("fp8 read back every byte")
    s = torch.tensor([[0.75], [3.0]], device="cuda")
    y = host(B().aq_fp8_dequantize(codes, s).double()).reshape(-1)
    ref = O.decode(np.arange(256)) * np.repeat([0.75, 3.0], 128)
    assert (np.nan_to_num(y, nan=-1) == np.nan_to_num(ref, nan=-1)).all()


def test_stacks_and_strides():
    rng = np.random.default_rng(9)
    step("fp8 quantize stacks and strided rows")
    w = _input(rng, 3, 150, 272)
    pair = B().aq_fp8_quantize(dev(w), 128)
    assert tuple(pair[1].shape) == (3, 2, 3)
    _same(pair, O.quantize(w, 128), "stack")
    y = B().aq_fp8_dequantize(*pair, 128)
    assert (host(y) == O.dequantize(_bytes(pair[0]), host(pair[1])).astype(np.float32)).all()
    base = dev(_input(rng, 40, 320))
    for x in (base[:, 16:288], base[1::2, :48], base[:1, 32:96], base.view(4, 10, 320)[:, :, :256]):
        for br in (1, 128):
            got, ref = B().aq_fp8_quantize(x, br), B().aq_fp8_quantize(x.contiguous(), br)
            assert torch.equal(got[0].view(torch.uint8), ref[0].view(torch.uint8)) and torch.equal(got[1], ref[1])
    for bad in (base.t(), base[:, ::2], base[:, :40], base[:, 2:50], base[0].expand(5, 320), base.view(4, 10, 320)[:, :9]):
        with pytest.raises(ValueError):
            B().aq_fp8_quantize(bad)
    empty = B().aq_fp8_quantize(base[:0])
    assert tuple(empty[0].shape) == (0, 320) and tuple(empty[1].shape) == (0, 3)


def test_outputs_given_streams_and_refusals():
    x = torch.randn(33, 256, device="cuda")
    codes, scales = torch.empty(33, 256, dtype=torch.uint8, device="cuda"), torch.empty(33, 2, device="cuda")
    ref = B().aq_fp8_quantize(x)
    step("fp8 quantize into given outputs on a side stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = B().aq_fp8_quantize(x, codes=codes, scales=scales)
    side.synchronize()
    assert got[0] is codes and got[1] is scales
    assert torch.equal(codes, ref[0].view(torch.uint8)) and torch.equal(scales, ref[1])
    for kw in (dict(codes=codes[:32]), dict(codes=codes.float()), dict(scales=scales.double()), dict(scales=scales.t())):
        with pytest.raises(ValueError):
            B().aq_fp8_quantize(x, **kw)
    for args in ((codes.float(), scales), (codes, scales[:, :1].contiguous()), (codes, scales, 128), (codes, scales, 1, torch.float16)):
        with pytest.raises(ValueError):
            B().aq_fp8_dequantize(*args)
    with pytest.raises(ValueError, match="block_rows"):
        B().aq_fp8_quantize(x, 64)
    with pytest.raises(ValueError):
        B().aq_fp8_quantize(x.half())


def test_more_elements_than_32_bits_count():
    """2^32 + 2^20 elements: the first and last rows against slices of their own."""
    k = 4096
    m = (1 << 20) + 256
    x = torch.empty(m, k, dtype=BF16, device="cuda")
    x[:300].normal_()
    x[300:-300] = 1.0
    x[-300:].normal_()
    step("fp8 quantize 2^32 + 2^20 elements")
    for br in (1, 128):
        c, s = B().aq_fp8_quantize(x, br)
        last = m - 256
        cl, sl = B().aq_fp8_quantize(x[last:].clone(), br)
        assert torch.equal(c[last:].view(torch.uint8), cl.view(torch.uint8)) and torch.equal(s[last // br:], sl)
        y = B().aq_fp8_dequantize(c, s, br, out_dtype=BF16)
        assert torch.equal(y[last:], B().aq_fp8_dequantize(cl, sl, br, out_dtype=BF16))
        assert (y[m // 2] == 1.0).all()
        del c, s, y
