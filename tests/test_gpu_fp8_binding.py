"""The FP8 and routing calls through the binding's native module and step by step give the same tensors and the same errors."""
import pytest
import torch

from tests.gpu_util import step

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


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
    x = torch.randn(5, 144, device="cuda", generator=g)
    xb, wide = x.bfloat16(), torch.randn(5, 304, device="cuda", generator=g).bfloat16()
    w = torch.randn(3, 260, 144, device="cuda", generator=g)
    wc, ws = B.aq_fp8_quantize(w, 128)
    off, rows = torch.tensor([0, 2, 2, 6], device="cuda", dtype=torch.int32), torch.tensor([4, 0, 0, 1, 2, 3], device="cuda",
                                                                                           dtype=torch.int32)
    off5 = torch.tensor([0, 3, 3, 5], device="cuda", dtype=torch.int32)
    q = B.aq_fp8_quantize(xb)
    qb = q[0].view(torch.uint8), q[1]
    out = torch.zeros(5, 260, device="cuda", dtype=BF16)
    logits = torch.randn(7, 24, device="cuda", generator=g)
    bias = torch.randn(24, device="cuda", generator=g)
    ids, weights = B.aq_moe_route(logits, 3)
    dw = torch.randn(7, 3, device="cuda", generator=g)
    dc, ds = B.aq_fp8_quantize(torch.randn(3, 144, 128, device="cuda", generator=g), 128)
    gc, gs = wc[:, :256].contiguous(), ws[:, :2].contiguous()
    choice = torch.randint(-1, 4, (5, 2), device="cuda", generator=g).int()
    cw = torch.rand(5, 2, device="cuda", generator=g)
    yield "quantize f32", lambda: B.aq_fp8_quantize(x)
    yield "quantize bf16 rows apart", lambda: B.aq_fp8_quantize(wide[:, 32:176])
    yield "quantize one row", lambda: B.aq_fp8_quantize(wide[:1, 64:])
    yield "quantize blocks", lambda: B.aq_fp8_quantize(w[1], 128)
    yield "quantize a stack", lambda: B.aq_fp8_quantize(w, block_rows=128)
    yield "dequantize", lambda: B.aq_fp8_dequantize(*q)
    yield "dequantize bytes to bf16", lambda: B.aq_fp8_dequantize(*qb, out_dtype=BF16)
    yield "dequantize blocks", lambda: B.aq_fp8_dequantize(wc[2], ws[2], 128)
    yield "dequantize a stack", lambda: B.aq_fp8_dequantize(wc, ws, block_rows=128)
    yield "gemm", lambda: B.aq_fp8_gemm(*q, wc[1], ws[1])
    yield "gemm out", lambda: B.aq_fp8_gemm(*qb, wc[0], ws[0], out=out)
    yield "linear", lambda: B.aq_fp8_linear(xb, wc[1], ws[1], out_dtype=BF16)
    yield "linear f32 rows apart", lambda: B.aq_fp8_linear(wide.float()[:, 32:176], wc[0], ws[0])
    yield "linear out", lambda: B.aq_fp8_linear(x, wc[0], ws[0], out=out)
    yield "grouped", lambda: B.aq_fp8_grouped_gemm(*q, wc, ws, off, rows)[:6]
    yield "grouped without rows", lambda: B.aq_fp8_grouped_gemm(*q, wc, ws, off5, out_dtype=BF16)
    for score in ("softmax", "sigmoid"):
        yield "route " + score, lambda: B.aq_moe_route(logits, 3, score=score)
        yield "route with bias and groups " + score, lambda: B.aq_moe_route(logits, 4, score=score, bias=bias, groups=4, top_groups=2, renormalize=False,
                                                                            scale=2)
        yield "route backward " + score, lambda: B.aq_moe_route_backward(logits, ids, weights, dw, score=score, scale=0.5)
    yield "route rows apart", lambda: B.aq_moe_route(wide[:, 3:200], 5)
    yield "experts", lambda: B.aq_fp8_experts(xb, gc, gs, dc, ds, choice, cw)[::2]
    yield "experts bf16", lambda: B.aq_fp8_experts(x, gc, gs, dc, ds, choice, cw, BF16)[::2]
    yield "no rows", lambda: B.aq_fp8_linear(xb[:0], wc[0], ws[0])
    yield "no tokens", lambda: B.aq_moe_route(logits[:0], 3)
    yield "parameter", lambda: B.aq_fp8_quantize(torch.nn.Parameter(x))


def test_native_and_stepwise_calls_agree(monkeypatch):
    from weight_only_bit_group_amd import binding as B
    step("FP8 and routing calls, native")
    native = {}
    for name, call in _calls(B):
        y = call()
        native[name] = [t.clone() for t in (y if isinstance(y, tuple) else (y,))]
    monkeypatch.setattr(B, "_mx", _Refuses())
    step("FP8 and routing calls, step by step")
    for name, call in _calls(B):
        y = call()
        y = y if isinstance(y, tuple) else (y,)
        assert [(t.dtype, t.shape, t.device) for t in y] == [(t.dtype, t.shape, t.device) for t in native[name]], name
        assert all(torch.equal(a.view(torch.uint8) if a.dtype == F8 else a, b.view(torch.uint8) if b.dtype == F8 else b)
                   for a, b in zip(y, native[name])), name


def test_native_calls_return_the_output_given():
    from weight_only_bit_group_amd import binding as B
    x, w = torch.randn(3, 64, device="cuda").bfloat16(), torch.randn(8, 64, device="cuda")
    c, s = B.aq_fp8_quantize(w, 128)
    out = torch.empty(3, 8, device="cuda", dtype=BF16)
    assert B.aq_fp8_linear(x, c, s, out=out) is out
    assert torch.equal(out, B.aq_fp8_linear(x, c, s, BF16))
    codes, scales = torch.empty(3, 64, device="cuda", dtype=F8), torch.empty(3, 1, device="cuda")
    got = B.aq_fp8_quantize(x, codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales
    assert torch.equal(B.aq_fp8_quantize(x)[1], scales)


def test_native_calls_run_on_the_current_stream():
    """Work queued on a side stream before and after the calls: they take their place between."""
    from weight_only_bit_group_amd import binding as B
    c, s = B.aq_fp8_quantize(torch.randn(512, 2048, device="cuda"), 128)
    x = torch.zeros(64, 2048, device="cuda", dtype=BF16)
    one = torch.ones_like(x)
    ref, rid = B.aq_fp8_linear(one, c, s), B.aq_moe_route(one[:, :16], 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            x.fill_(float("nan"))
            big = torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
            x.copy_(one)
            y, r = B.aq_fp8_linear(x, c, s), B.aq_moe_route(x[:, :16], 2)
            x.zero_()
        side.synchronize()
        assert torch.equal(y, ref) and torch.equal(r[1], rid[1]) and big.shape == (4096, 4096)


def test_errors_come_through():
    from weight_only_bit_group_amd import binding as B
    x, w = torch.randn(3, 64, device="cuda").bfloat16(), torch.randn(8, 64, device="cuda")
    c, s = B.aq_fp8_quantize(w, 128)
    l = torch.randn(4, 8, device="cuda")
    for what, call in (("block_rows", lambda: B.aq_fp8_quantize(x, 64)), ("scales must be", lambda: B.aq_fp8_linear(x, c, s[:0])),
                       ("out_dtype", lambda: B.aq_fp8_linear(x, c, s, torch.float16)),
                       ("Y must be", lambda: B.aq_fp8_linear(x, c, s, BF16, out=torch.empty(3, 8, device="cuda"))),
                       ("ldx", lambda: B.aq_fp8_linear(torch.zeros(3, 66, device="cuda", dtype=BF16)[:, :64], c, s)),
                       ("aligned", lambda: B.aq_fp8_quantize(torch.zeros(200, device="cuda", dtype=BF16)[4:196].view(3, 64))),
                       ("GPU tensor", lambda: B.aq_fp8_linear(x.cpu(), c, s)), ("multiple of 16", lambda: B.aq_fp8_quantize(x[:, :8])),
                       ("top must be", lambda: B.aq_moe_route(l, 9)), ("score", lambda: B.aq_moe_route(l, 2, score="tanh")),
                       ("groups", lambda: B.aq_moe_route(l, 2, groups=3)), ("top_groups", lambda: B.aq_moe_route(l, 3, groups=4, top_groups=1)),
                       ("bias", lambda: B.aq_moe_route(l, 2, bias=l[0].double())), ("scale", lambda: B.aq_moe_route(l, 2, scale=float("inf")))):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError):
        B.aq_fp8_quantize(None)
