"""The MXFP4 calls through the binding's native module and step by step give the same tensors and the same errors."""
import pytest
import torch

from tests.gpu_util import step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class _Refuses:
    """Stands for the native module: every call goes through the binding's own steps."""

    def __getattr__(self, name):
        return lambda *a: None


def _calls(B):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(5, 96, device="cuda", generator=g)
    xb, wide = x.bfloat16(), torch.randn(5, 160, device="cuda", generator=g).bfloat16()
    wc = torch.randint(0, 256, (2, 24, 48), device="cuda", generator=g, dtype=torch.uint8)
    ws = torch.randint(120, 130, (2, 24, 3), device="cuda", generator=g, dtype=torch.uint8)
    off, rows = torch.tensor([0, 2, 6], device="cuda", dtype=torch.int32), torch.tensor([4, 0, 0, 1, 2, 3], device="cuda",
                                                                                         dtype=torch.int32)
    off5 = torch.tensor([0, 3, 5], device="cuda", dtype=torch.int32)
    q = B.aq_mxfp4_quantize(xb)
    out = torch.zeros(5, 24, device="cuda", dtype=torch.bfloat16)
    yield "quantize f32", lambda: B.aq_mxfp4_quantize(x)
    yield "quantize bf16 rows apart", lambda: B.aq_mxfp4_quantize(wide[:, 32:128])
    yield "quantize one row", lambda: B.aq_mxfp4_quantize(wide[:1, 64:])
    yield "dequantize", lambda: B.aq_mxfp4_dequantize(*q)
    yield "dequantize bf16", lambda: B.aq_mxfp4_dequantize(*q, out_dtype=torch.bfloat16)
    yield "gemm", lambda: B.aq_mxfp4_gemm(xb, wc[1], ws[1])
    yield "gemm rows apart", lambda: B.aq_mxfp4_gemm(wide[:, 32:128], wc[0], ws[0], torch.bfloat16)
    yield "gemm out", lambda: B.aq_mxfp4_gemm(xb, wc[0], ws[0], out=out)
    yield "gemm_a4", lambda: B.aq_mxfp4_gemm_a4(*q, wc[0], ws[0], out_dtype=torch.float32)
    yield "grouped", lambda: B.aq_mxfp4_grouped_gemm(xb, wc, ws, off, rows)
    yield "grouped without rows", lambda: B.aq_mxfp4_grouped_gemm(xb, wc, ws, off5, out_dtype=torch.bfloat16)
    yield "grouped_a4", lambda: B.aq_mxfp4_grouped_gemm_a4(*q, wc, ws, off, rows=rows)
    yield "no rows", lambda: B.aq_mxfp4_gemm(xb[:0], wc[0], ws[0])
    yield "parameter", lambda: B.aq_mxfp4_quantize(torch.nn.Parameter(x))


def test_native_and_stepwise_calls_agree(monkeypatch):
    from weight_only_bit_group_amd import binding as B
    step("MXFP4 calls, native")
    native = {name: call() for name, call in _calls(B)}
    native = {k: [t.clone() for t in v] if isinstance(v, tuple) else [v.clone()] for k, v in native.items()}
    monkeypatch.setattr(B, "_mx", _Refuses())
    step("MXFP4 calls, step by step")
    for name, call in _calls(B):
        y = call()
        y = list(y) if isinstance(y, tuple) else [y]
        assert [(t.dtype, t.shape, t.device) for t in y] == [(t.dtype, t.shape, t.device) for t in native[name]], name
        assert all(torch.equal(a, b) for a, b in zip(y, native[name])), name


def test_native_calls_return_the_output_given():
    from weight_only_bit_group_amd import binding as B
    x, w = torch.randn(3, 64, device="cuda").bfloat16(), torch.randn(8, 64, device="cuda")
    c, s = B.aq_mxfp4_quantize(w)
    out = torch.empty(3, 8, device="cuda", dtype=torch.bfloat16)
    assert B.aq_mxfp4_gemm(x, c, s, out=out) is out
    assert torch.equal(out, B.aq_mxfp4_gemm(x, c, s, torch.bfloat16))


def test_native_calls_run_on_the_current_stream():
    """Work queued on a side stream before and after the call: the call takes its place between."""
    from weight_only_bit_group_amd import binding as B
    w = torch.randn(512, 2048, device="cuda")
    c, s = B.aq_mxfp4_quantize(w)
    x = torch.zeros(64, 2048, device="cuda", dtype=torch.bfloat16)
    one = torch.ones_like(x)
    ref = B.aq_mxfp4_gemm(one, c, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            x.zero_()
            big = torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
            x.copy_(one)
            y = B.aq_mxfp4_gemm(x, c, s)
            x.zero_()
        side.synchronize()
        assert torch.equal(y, ref) and big.shape == (4096, 4096)


def test_errors_come_through():
    from weight_only_bit_group_amd import binding as B
    x, w = torch.randn(3, 64, device="cuda").bfloat16(), torch.randn(8, 64, device="cuda")
    c, s = B.aq_mxfp4_quantize(w)
    with pytest.raises(ValueError, match="scales must be"):
        B.aq_mxfp4_gemm(x, c, s[:4])
    with pytest.raises(ValueError, match="out_dtype"):
        B.aq_mxfp4_gemm(x, c, s, torch.float16)
    with pytest.raises(ValueError, match="Y must be"):
        B.aq_mxfp4_gemm(x, c, s, torch.bfloat16, out=torch.empty(3, 8, device="cuda"))
    with pytest.raises(ValueError, match="ldx"):   # rows 132 bytes apart
        B.aq_mxfp4_gemm(torch.zeros(3, 66, device="cuda", dtype=torch.bfloat16)[:, :64], c, s)
    with pytest.raises(ValueError, match="aligned"):
        B.aq_mxfp4_gemm(torch.zeros(200, device="cuda", dtype=torch.bfloat16)[4:196].view(3, 64), c, s)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.aq_mxfp4_gemm(x.cpu(), c, s)
    with pytest.raises(TypeError):
        B.aq_mxfp4_quantize(None)
