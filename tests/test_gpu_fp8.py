"""FP8 products on the GPU against the 64-bit oracle.

The factors of a product have four significant bits each, so products are exact; a sum of K of them in fp32, in any
order and with each addition rounded or cut (a relative 2^-23 at most), is off by at most K 2^-23 sum |x w|, a
block's factor and its products by 2^-23 together.  With bf16 outputs every product of eight neighbouring k may lose
less than 2^-13 of the largest of the eight, all of them 2^-10 of it, and that is at most the product of the largest
factors; the rounding to bf16 adds at most 2^-8 of the value.  Inputs whose sums fit 24 bits, with scales that are
powers of two and products within 2^13 of each other, are compared for equality.
"""
import numpy as np
import pytest
import torch

from oracle import fp8 as O
from tests.gpu_util import dev, host, step

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def B():
    from weight_only_bit_group_amd import binding
    return binding


def _np(t):
    return host(t.double())


def _codes(rng, *shape):
    c = rng.integers(0, 254, shape, dtype=np.uint8)
    return c + (c >= 127)   # every byte but the two NaN


def _pair(rng, *shape, block_rows):
    s = np.exp(rng.standard_normal(O.scale_shape(shape, block_rows)) * 3).astype(np.float32)
    return _codes(rng, *shape), s


def _d(pair):
    return dev(pair[0]).view(F8), dev(pair[1])


def _eights(v):
    """The largest magnitude of every eight neighbouring k."""
    return np.abs(v).reshape(*v.shape[:-1], v.shape[-1] // 8, 8).max(-1)


def _bound(x, w, k):
    """{output type: how far the values of x w^T may be off before they are rounded to it}; x, w 64-bit values."""
    wide = (k + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    return {F32: wide, BF16: wide + 2.0 ** -10 * (_eights(x) @ _eights(w).T)}


def _close(y, ref, bound, what):
    tol = bound[y.dtype]
    if y.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(_np(y) - ref)
    print(f"[gpu] {what}: worst share of the bound {np.max(err / (tol + 1e-300)):.3f}", flush=True)
    assert (err <= tol).all(), what


SIZES = [(1, 1, 16), (1, 64, 128), (1, 1003, 2048), (2, 130, 144), (3, 127, 112), (5, 129, 272), (16, 256, 1024),
         (17, 100, 2064), (33, 300, 400), (64, 128, 128), (65, 129, 384), (100, 1, 640), (127, 500, 1040), (130, 257, 256),
         (257, 513, 512), (300, 1003, 2064)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm(m, n, k):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    x, w = _pair(rng, m, k, block_rows=1), _pair(rng, n, k, block_rows=128)
    ref, bound = O.forward(x, w), _bound(O.dequantize(*x), O.dequantize(*w), k)
    step(f"fp8 gemm {m} x {n} x {k}")
    for dtype in (F32, BF16):
        y = B().aq_fp8_gemm(*_d(x), *_d(w), out_dtype=dtype)
        assert y.dtype == dtype and tuple(y.shape) == (m, n)
        _close(y, ref, bound, f"{m} x {n} x {k} {dtype}")


@pytest.mark.parametrize("m,n,k", [(1, 300, 2064), (9, 257, 400), (70, 640, 1040), (300, 130, 272), (520, 1030, 384)])
def test_gemm_of_integers_is_exact(m, n, k):
    """Codes of -8 .. 8 and block scales of powers of two over a few bits: every sum fits 24 bits."""
    rng = np.random.default_rng(k)
    xv, wv = rng.integers(-8, 9, (m, k)), rng.integers(-8, 9, (n, k))
    x = O.encode(xv), np.exp2(rng.integers(-1, 2, O.scale_shape((m, k), 1))).astype(np.float32)
    w = O.encode(wv), np.exp2(rng.integers(-1, 2, O.scale_shape((n, k), 128))).astype(np.float32)
    step(f"fp8 gemm of integers {m} x {n} x {k}")
    ref = O.forward(x, w)
    assert (_np(B().aq_fp8_gemm(*_d(x), *_d(w))) == ref).all()
    assert (_np(B().aq_fp8_gemm(*_d(x), *_d(w), out_dtype=BF16)) == host(torch.from_numpy(ref).to(BF16).double())).all()


def _large(rng, m, n, k):
    """Inputs made on the device and the result in 64 bits there (float64 products of the dequantized values)."""
    g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
    x = B().aq_fp8_quantize(torch.randn(m, k, generator=g, device="cuda"))
    w = B().aq_fp8_quantize(torch.randn(n, k, generator=g, device="cuda"), 128)
    xv = B().aq_fp8_dequantize(*x).double()
    wv = B().aq_fp8_dequantize(*w, 128).double()
    return x, w, xv, wv


@pytest.mark.parametrize("m,n,k", [(1, 11008, 2048), (16, 4096, 14336), (48, 2048, 4096), (512, 2048, 2048), (1000, 4096, 1040),
                                   (4096, 2176, 2048), (2500, 11008, 528), (40, 300, 32768)])
def test_large_gemm(m, n, k):
    x, w, xv, wv = _large(np.random.default_rng(n), m, n, k)
    step(f"fp8 gemm {m} x {n} x {k}")
    ref = xv @ wv.t()
    # (xv and wv are rounded to fp32: 2^-24 each)
    tol = (k + 6) * 2.0 ** -23 * (xv.abs() @ wv.abs().t())
    y = B().aq_fp8_gemm(*x, *w)
    assert ((y.double() - ref).abs() <= tol).all()
    tol += 2.0 ** -10 * (xv.abs().unflatten(1, (-1, 8)).amax(2) @ wv.abs().unflatten(1, (-1, 8)).amax(2).t())
    y = B().aq_fp8_gemm(*x, *w, out_dtype=BF16)
    assert ((y.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all()


def test_rows_do_not_depend_on_one_another_and_calls_repeat():
    rng = np.random.default_rng(4)
    x, w = _d(_pair(rng, 40, 400, block_rows=1)), _d(_pair(rng, 300, 400, block_rows=128))
    step("fp8 gemm, a row of NaN beside others, twice")
    y = B().aq_fp8_gemm(*x, *w)
    assert torch.equal(y, B().aq_fp8_gemm(*x, *w))
    bad = x[0].clone().view(torch.uint8), x[1].clone()
    bad[0][7, 3] = 127
    bad[1][11, 2] = float("nan")
    z = B().aq_fp8_gemm(*bad, *w)
    rows = [r for r in range(40) if r not in (7, 11)]
    assert torch.equal(z[rows], y[rows]) and z[7].isnan().all() and z[11].isnan().all()
    bad = w[0].clone().view(torch.uint8), w[1].clone()
    bad[0][130, 399] = 255
    bad[1][2, 0] = float("inf")
    z = B().aq_fp8_gemm(*x, *bad)
    cols = [c for c in range(256) if c != 130]
    assert torch.equal(z[:, cols], y[:, cols]) and z[:, 130].isnan().all() and not z[:, 256:].isfinite().any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 300, 2064), (4, 64, 16), (16, 200, 2048), (33, 129, 144), (300, 257, 1040), (1000, 520, 400)])
def test_linear_is_quantise_and_gemm(m, n, k, dtype):
    rng = np.random.default_rng(m + n)
    x = dev((rng.standard_normal((m, k)) * 2).astype(np.float32)).to(dtype)
    if m > 2:
        x[1, 5] = float("nan")
    w = _d(_pair(rng, n, k, block_rows=128))
    step(f"fp8 linear {m} x {n} x {k} {dtype}")
    for out in (F32, BF16):
        ref = B().aq_fp8_gemm(*B().aq_fp8_quantize(x), *w, out_dtype=out)
        y = B().aq_fp8_linear(x, *w, out_dtype=out)
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(ref)) and torch.equal(y.isnan(), ref.isnan())
    ws = torch.empty(B().aq_fp8_linear_workspace(m, k), dtype=torch.uint8, device="cuda")
    given = torch.empty(m, n, device="cuda")
    wide = torch.zeros(m, k + 32, dtype=dtype, device="cuda")
    wide[:, 16:16 + k] = x
    assert B().aq_fp8_linear(wide[:, 16:16 + k], *w, out=given, workspace=ws) is given
    assert torch.equal(torch.nan_to_num(given), torch.nan_to_num(B().aq_fp8_linear(x, *w)))


# ---- grouped by expert -------------------------------------------------------------------------------

GROUPED = [([0, 1], None, 64, 128), ([0, 3, 3, 8], None, 130, 272), ([0, 0, 0, 5], 7, 100, 144), ([2, 20, 20, 37, 90], 40, 257, 400),
           ([0, 200, 201, 500], 64, 129, 1040), ([5, 700], 300, 300, 256), ([0] + list(range(3, 300, 3)), 50, 70, 112)]


@pytest.mark.parametrize("offsets,t,n,k", GROUPED)
def test_grouped(offsets, t, n, k):
    rng = np.random.default_rng(n + k)
    e, m = len(offsets) - 1, offsets[-1] + 3
    rows = None if t is None else rng.integers(0, t, m).astype(np.int32)
    x, w = _pair(rng, m if t is None else t, k, block_rows=1), _pair(rng, e, n, k, block_rows=128)
    off = np.array(offsets, np.int32)
    ref = O.grouped_forward(x, w, off, rows)
    xv, wv = O.dequantize(*x), O.dequantize(*w)
    xv = xv if rows is None else xv[rows]
    bound = {F32: np.zeros(ref.shape), BF16: np.zeros(ref.shape)}
    for i in range(e):
        part = slice(off[i], off[i + 1])
        for dtype, b in _bound(xv[part], wv[i], k).items():
            bound[dtype][part] = b
    step(f"fp8 grouped gemm {offsets[:6]} rows of {t}, {n} x {k}")
    inside = slice(offsets[0], offsets[-1])
    for dtype in (F32, BF16):
        y = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
        B().aq_fp8_grouped_gemm(*_d(x), *_d(w), dev(off), None if rows is None else dev(rows), out=y)
        _close(y[inside], ref[inside], {dtype: bound[dtype][inside]}, f"grouped {dtype}")
        assert (y[:offsets[0]] == 7).all() and (y[offsets[-1]:] == 7).all()


def test_grouped_equals_the_dense_product():
    """Every expert's rows against the dense product with its weights: the same bits where the same kernel runs, and
    within the bound where it does not."""
    rng = np.random.default_rng(12)
    e, n, k = 6, 384, 528
    counts = [0, 1, 17, 300, 64, 130]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, w = _pair(rng, off[-1], k, block_rows=1), _pair(rng, e, n, k, block_rows=128)
    step("fp8 grouped against dense")
    y = _np(B().aq_fp8_grouped_gemm(*_d(x), *_d(w), dev(off)))
    for i in range(e):
        part = slice(off[i], off[i + 1])
        if counts[i]:
            one, wi = (x[0][part], x[1][part]), (w[0][i], w[1][i])
            z = _np(B().aq_fp8_gemm(*_d(one), *_d(wi)))
            assert (np.abs(z - y[part]) <= 2 * _bound(O.dequantize(*one), O.dequantize(*wi), k)[F32]).all()


@pytest.mark.parametrize("m", [6, 90, 700])
def test_lists_that_lead_nowhere(m):
    """Rows outside X become NaN, offsets outside 0 .. M are clamped, an expert that ends before it starts is empty."""
    rng = np.random.default_rng(m)
    t, n, k = 9, 150, 272
    x, w = _pair(rng, t, k, block_rows=1), _pair(rng, 3, n, k, block_rows=128)
    rows = rng.integers(0, t, m).astype(np.int32)
    bad = rng.permutation(m)[:m // 3]
    rows[bad] = rng.choice([-1, t, 2 ** 31 - 1, -2 ** 31], len(bad))
    step(f"fp8 grouped with lists outside their range, {m} rows")
    half = m // 2
    for off in ([0, half, half, m], [-5, half, half, m + 100], [-2 ** 31, half, half - 1, 2 ** 31 - 1]):
        lo = np.array(off, np.int32)
        y = _np(B().aq_fp8_grouped_gemm(*_d(x), *_d(w), dev(lo), dev(rows)))
        assert np.isnan(y[bad]).all()
        good = np.setdiff1d(np.arange(m), bad)
        # (in the last list the middle rows are claimed twice: only the first expert's are compared)
        for r in good[good < half - 1]:
            one, w0 = O.dequantize(x[0][rows[r]][None], x[1][rows[r]][None]), O.dequantize(w[0][0], w[1][0])
            assert (np.abs(y[r] - (one @ w0.T)[0]) <= _bound(one, w0, k)[F32][0]).all()
    y = torch.full((m, n), 3.0, device="cuda")
    B().aq_fp8_grouped_gemm(*_d(x), *_d(w), dev(np.array([9, 7, 5, 3], np.int32)), dev(rows), out=y)
    assert (y == 3).all()


def test_grouped_follows_its_lists_when_replayed():
    rng = np.random.default_rng(2)
    x, w = _d(_pair(rng, 30, 400, block_rows=1)), _d(_pair(rng, 4, 200, 400, block_rows=128))
    off, rows = dev(np.array([0, 5, 9, 30, 64], np.int32)), dev(rng.integers(0, 30, 64).astype(np.int32))
    step("fp8 grouped captured and replayed")
    y = torch.zeros(64, 200, device="cuda")
    B().aq_fp8_grouped_gemm(*x, *w, off, rows, out=y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B().aq_fp8_grouped_gemm(*x, *w, off, rows, out=y)
    for lists in ([0, 5, 9, 30, 64], [0, 0, 64, 64, 64], [1, 2, 3, 4, 60]):
        off.copy_(torch.tensor(lists, dtype=torch.int32))
        rows.copy_(torch.randint(0, 30, (64,), dtype=torch.int32))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        z = torch.zeros_like(y)
        B().aq_fp8_grouped_gemm(*x, *w, off, rows, out=z)
        assert torch.equal(y, z)


def test_linear_captured_and_replayed():
    rng = np.random.default_rng(8)
    w = _d(_pair(rng, 256, 528, block_rows=128))
    step("fp8 linear captured and replayed")
    for m in (1, 16, 200):
        x = torch.randn(m, 528, device="cuda").to(BF16)
        y = B().aq_fp8_linear(x, *w)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            z = B().aq_fp8_linear(x, *w)
        for _ in range(3):
            x.normal_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(z, B().aq_fp8_linear(x, *w))


def test_refusals():
    rng = np.random.default_rng(1)
    x, w = _d(_pair(rng, 8, 256, block_rows=1)), _d(_pair(rng, 200, 256, block_rows=128))
    e = w[0][None], w[1][None]
    off = dev(np.array([0, 8], np.int32))
    step("fp8 product refusals")
    for bad in ((x[0][:, :128], x[1], *w), (x[0], x[1][:, :1].contiguous(), *w), (x[0].float(), x[1], *w), (x[0], x[1].half(), *w),
                (*x, w[0][:, :240].contiguous(), w[1]), (*x, w[0], w[1][:1].contiguous()), (*x, *e), (x[0][None], x[1], *w)):
        with pytest.raises(ValueError):
            B().aq_fp8_gemm(*bad)
    for kw in (dict(out_dtype=torch.float16), dict(out=torch.empty(8, 199, device="cuda")),
               dict(out=torch.empty(8, 200, device="cuda"), out_dtype=BF16)):
        with pytest.raises(ValueError):
            B().aq_fp8_gemm(*x, *w, **kw)
    for bad in ((*x, *w, off), (*x, *e, off.long()), (*x, *e, off[:1]), (*x, *e, off, off.long()), (*x, *e, off, off[None])):
        with pytest.raises(ValueError):
            B().aq_fp8_grouped_gemm(*bad)
    xf = torch.randn(8, 256, device="cuda")
    for bad in (xf.half(), xf[:, :200], xf.t(), xf[None]):
        with pytest.raises(ValueError):
            B().aq_fp8_linear(bad, *w)
    with pytest.raises(ValueError, match="workspace"):
        B().aq_fp8_linear(xf, *w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert B().aq_fp8_gemm(x[0][:0], x[1][:0], *w).shape == (0, 200)
    assert B().aq_fp8_linear(xf[:0], *w).shape == (0, 200)
    assert B().aq_fp8_gemm(*x, w[0][:0], w[1][:0]).shape == (8, 0)
