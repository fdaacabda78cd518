"""Refusals of the MXFP4 modules that need no GPU."""
import pytest
import torch

from weight_only_bit_group_amd import layer as L

U8 = torch.uint8


def _pair(*lead, k=64):
    return torch.zeros(*lead, k // 2, dtype=U8), torch.zeros(*lead, k // 32, dtype=U8)


def test_linear_refuses_wrong_buffers():
    c, s = _pair(8)
    L.MXFP4Linear(c, s)
    for bad in ((c.int(), s), (c, s.float()), (c[0], s), (c, s[:4]), (c[:, :24], s), (c[:, :0], s[:, :0]), (c, s, None, "fp8")):
        with pytest.raises(ValueError):
            L.MXFP4Linear(*bad)


def test_experts_refuse_wrong_buffers():
    gu, d = _pair(3, 128, k=96), _pair(3, 96, k=64)
    m = L.MXFP4Experts(*gu, *d)
    assert (m.num_experts, m.features, m.inner) == (3, 96, 64)
    for bad in ((*gu, *_pair(3, 64, k=64)), (*gu, *_pair(2, 96, k=64)), (*gu, *_pair(3, 96, k=96)), (*_pair(384, k=96), *d),
                (*gu, d[0], d[1][..., :1]), (*gu, *d, "int8")):
        with pytest.raises(ValueError):
            L.MXFP4Experts(*bad)


def test_quantized_linear_is_not_quantized_again():
    model = torch.nn.ModuleDict({"a": L.MXFP4Linear(*_pair(8)), "b": torch.nn.Linear(64, 8)})
    with pytest.raises(ValueError, match="already quantized: a"):
        L.plan_quantization(model, ("a", "b"))
    assert list(L.plan_quantization(model, ("b",))) == ["b"]
    with pytest.raises(ValueError, match="already quantized"):
        L.quantize_linear(model["a"], 64)


def test_weights_on_the_host_are_refused():
    with pytest.raises(ValueError, match="GPU tensor"):
        L.MXFP4Linear.from_weight(torch.zeros(8, 64))
    with pytest.raises(ValueError, match="3 dimensions"):
        L.MXFP4Experts.from_weights(torch.zeros(8, 64), torch.zeros(2, 64, 32))


def _with_products_on_the_host(monkeypatch):
    """The binding's calls of the modules replaced by plain ones (values as dequantized by the oracle)."""
    import numpy as np

    from oracle import mxfp4 as O

    def weight(codes, scales):
        return torch.from_numpy(np.asarray(O.dequantize(codes.numpy(), scales.numpy()))).float()

    def gemm(x, codes, scales):
        return x.detach().float() @ weight(codes, scales).t()

    def grouped(x, codes, scales, offsets, rows=None):
        w, x = weight(codes, scales), x.detach().float()
        x = x if rows is None else x[rows.long()]
        y = torch.zeros(x.shape[0], w.shape[1])
        for e in range(w.shape[0]):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            y[lo:hi] = x[lo:hi] @ w[e].t()
        return y

    monkeypatch.setattr(L.B, "aq_mxfp4_gemm", gemm)
    monkeypatch.setattr(L.B, "aq_mxfp4_grouped_gemm", grouped)


def _random_pair(g, *lead, k):
    return (torch.randint(0, 256, (*lead, k // 2), generator=g, dtype=U8),
            torch.randint(125, 129, (*lead, k // 32), generator=g, dtype=U8))


def test_linear_has_no_silent_gradient(monkeypatch):
    """The input's gradient is refused when it is asked for; the forward pass and what stands beside it are as ever."""
    _with_products_on_the_host(monkeypatch)
    g = torch.Generator().manual_seed(1)
    lin = L.MXFP4Linear(*_random_pair(g, 64, k=64), torch.ones(64))
    x = torch.randn(3, 2, 64, generator=g)
    plain = lin(x)
    assert not plain.requires_grad
    xg = x.clone().requires_grad_()
    y = lin(xg)
    assert torch.equal(y, plain) and y.requires_grad
    y += 1                                         # in place, as on any linear's output
    for loss in (y, xg + lin(xg)):                 # alone, and in a residual path
        with pytest.raises(RuntimeError, match="MXFP4Linear has no backward pass"):
            loss.sum().backward()
    with torch.no_grad():
        assert not lin(xg).requires_grad
    with torch.inference_mode():
        assert torch.equal(lin(x), plain)


def test_experts_have_no_silent_gradient(monkeypatch):
    """The gradient of the router's weights is the formula's; one that would pass through the experts is refused."""
    _with_products_on_the_host(monkeypatch)
    g = torch.Generator().manual_seed(2)
    m = L.MXFP4Experts(*_random_pair(g, 4, 64, k=64), *_random_pair(g, 4, 64, k=32))
    x, ids = torch.randn(5, 64, generator=g), torch.randint(0, 5, (5, 2), generator=g)   # (choice 4 adds nothing)
    ids[:, 1] = (ids[:, 0] + 1) % 5
    w = torch.rand(5, 2, generator=g)
    plain = m(x, ids, w)
    assert not plain.requires_grad
    wg, dy = w.clone().requires_grad_(), torch.randn(5, 64, generator=g)
    y = m(x, ids, wg)
    assert torch.equal(y, plain)
    y.backward(dy)
    for j in range(2):
        one = torch.zeros_like(w)
        one[:, j] = 1
        # 64 products and sums in fp32, each off by 2^-24 of the magnitudes at most
        part = m(x, ids, one)
        assert ((wg.grad[:, j] - (part * dy).sum(1)).abs() <= 65 * 2.0 ** -23 * (part * dy).abs().sum(1)).all()
    xg = x.clone().requires_grad_()
    router = torch.nn.Linear(64, 2)
    for residual in (False, True):
        y = m(xg, ids, router(xg))
        with pytest.raises(RuntimeError, match="MXFP4Experts has no backward pass"):
            (xg + y if residual else y).sum().backward()


def test_experts_refuse_a_capture_that_sorts_too_much(monkeypatch):
    """More than 2^20 choices in a captured call: the sort of so many is not repeated faithfully by a replay."""
    _with_products_on_the_host(monkeypatch)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    g = torch.Generator().manual_seed(4)
    m = L.MXFP4Experts(*_random_pair(g, 2, 64, k=32), *_random_pair(g, 2, 32, k=32))
    t = (1 << 18) + 1
    with pytest.raises(RuntimeError, match="choices in a captured call"):
        m(torch.zeros(t, 32), torch.zeros(t, 4, dtype=torch.int32), torch.zeros(t, 4))
    assert m(torch.zeros(5, 32), torch.zeros(5, 4, dtype=torch.int32), torch.zeros(5, 4)).shape == (5, 32)
