"""FP8 modules on the GPU: rounding, products, routing, experts and the sum over choices run together.

The first products' inputs are whole numbers that FP8 holds with the factor 1 (every block has a 448, those of the two
operands among different eights of k, so that no product is below 2^-13 of its neighbours'): gate and up values are
exact.  The activations between the products come from the kernel that is tested by itself, on the oracle's exact
values.  The second product then differs from its 64-bit value as the products' tests say, and the sum over a token's
choices by 2^-23 a choice; with bf16 outputs each choice's products are rounded to bf16 first.
"""
import numpy as np
import pytest
import torch

from oracle import fp8 as O
from oracle import moe as OM
from tests.gpu_util import dev, host, step
from tests.test_gpu_fp8 import _bound

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def L():
    from weight_only_bit_group_amd import layer
    return layer


def B():
    from weight_only_bit_group_amd import binding
    return binding


def _x(rng, *shape):
    """Whole numbers of -8 .. 8 with a 448 in front of every block of 128 k of a row."""
    v = rng.integers(-8, 9, shape)
    v[..., ::128] = 448
    return v.astype(np.float32)


def _w(rng, *shape):
    """The same with a 448 at the ninth (or, in a short last block, the ninth as well) k of a 128 x 128 block's first row."""
    v = rng.integers(-8, 9, shape)
    v[..., ::128, 8::128] = 448
    return v.astype(np.float32)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 256), (2, 3, 144), (40, 256), (300, 2064)])
def test_linear_of_integers_is_exact(shape, dtype, out):
    rng = np.random.default_rng(shape[-1] + len(shape))
    k, n = shape[-1], 197
    w, x, b = _w(rng, n, k), _x(rng, *shape), rng.integers(-9, 9, n).astype(np.float32)
    step(f"FP8Linear {shape} {dtype} {out}")
    lin = L().FP8Linear.from_weight(dev(w), dev(b), out)
    assert (lin.scales == 1).all()
    y = lin(dev(x).to(dtype))
    ref = x.astype(np.float64) @ w.T.astype(np.float64)
    ref = torch.from_numpy(ref).to(out).double().numpy() + b     # (in bf16: rounded, then the bias added in bf16)
    assert y.dtype == out and tuple(y.shape) == (*shape[:-1], n)
    assert (host(y.double()) == torch.from_numpy(ref).to(out).double().numpy()).all()
    state = {name: t.clone() for name, t in lin.state_dict().items()}
    other = L().FP8Linear(torch.zeros_like(lin.codes), torch.zeros_like(lin.scales), torch.zeros_like(lin.bias), out)
    other.load_state_dict(state)
    assert torch.equal(other(dev(x).to(dtype)), y)


def test_linear_takes_rows_of_any_layout():
    rng = np.random.default_rng(5)
    lin = L().FP8Linear.from_weight(dev(rng.standard_normal((40, 64)).astype(np.float32)))
    base = dev(rng.standard_normal((9, 130)).astype(np.float32)).to(BF16)
    step("FP8Linear over views")
    for x in (base[:, 3:67], base[:, 8:72], base[1:, :64], base[:1, :64].expand(7, 64), base.t()[:64].t().contiguous(),
              base.reshape(-1)[1:65], base[:0, :64], base[:, :64].half(), base[:, :64].double()):
        assert torch.equal(lin(x), lin(x.clone(memory_format=torch.contiguous_format)))
    assert lin(base[:0, :64]).shape == (0, 40)


def _experts_reference(x, w1, w2, ids, weights, out):
    """(values, how far they may be off) of the experts in 64 bits; x and w1 exact, w2 a pair of codes and scales."""
    t, top = ids.shape
    k, inner = w2[0].shape[1:]
    y, tol = np.zeros((t, k)), np.zeros((t, k))
    for e in range(len(w1)):
        for j in range(top):
            at = np.flatnonzero(ids[:, j] == e)
            if not len(at):
                continue
            h = dev((x[at].astype(np.float64) @ w1[e].T.astype(np.float64)).astype(np.float32))
            c, s = B().aq_fp8_swiglu_quantize(h)
            h = O.dequantize(host(c.view(torch.uint8)), host(s))
            w = O.dequantize(w2[0][e], w2[1][e])
            part = h @ w.T
            f = np.abs(weights[at, j].astype(np.float64))[:, None]
            y[at] += weights[at, j].astype(np.float64)[:, None] * part
            off = _bound(h, w, inner)[out]
            if out == BF16:
                off = off + 2.0 ** -8 * (np.abs(part) + off)
            tol[at] += f * (off + top * 2.0 ** -23 * (np.abs(part) + off))
    if out == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
    return y, tol


def _experts(rng, e, k, inner, out):
    w1 = _w(rng, e, 2 * inner, k)
    m = L().FP8Experts.from_weights(dev(w1), dev(rng.standard_normal((e, k, inner)).astype(np.float32)), out)
    assert (m.gate_up_scales == 1).all()
    return m, w1, (host(m.down_codes.view(torch.uint8)), host(m.down_scales))


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("t,top,e,k,inner", [(1, 2, 4, 64, 32), (1, 8, 16, 256, 96), (5, 1, 3, 144, 64), (33, 2, 5, 64, 160), (150, 4, 7, 128, 256),
                                             (400, 3, 4, 272, 144), (700, 2, 3, 256, 384)])
def test_experts(t, top, e, k, inner, out):
    rng = np.random.default_rng(t * 100 + e)
    x = _x(rng, t, k)
    ids = np.stack([rng.permutation(e)[:top] for _ in range(t)])
    weights = rng.random((t, top)).astype(np.float32)
    step(f"FP8Experts t {t} top {top} e {e} k {k} inner {inner} {out}")
    m, w1, w2 = _experts(rng, e, k, inner, out)
    y = m(dev(x).to(BF16), dev(ids), dev(weights))
    ref, tol = _experts_reference(x, w1, w2, ids, weights, out)
    err = np.abs(host(y.double()) - ref)
    print(f"[gpu] worst share of the bound {(err / (tol + 1e-300)).max():.3f}", flush=True)
    assert y.dtype == out and (err <= tol).all()


@pytest.mark.parametrize("ids_dtype", [torch.int64, torch.int32, torch.uint8])
def test_experts_with_choices_that_add_nothing(ids_dtype):
    """Choices outside the range, tokens without a valid one, an expert chosen twice by a token, and no tokens."""
    rng = np.random.default_rng(3)
    e, k, inner = 4, 64, 32
    x = _x(rng, 6, k)
    ids = np.array([[0, 1], [4, 4], [200, 2], [3, 3], [1, 99], [4, 0]])
    weights = rng.random((6, 2)).astype(np.float32)
    weights[(ids < 0) | (ids >= e)] = np.nan
    m, w1, w2 = _experts(rng, e, k, inner, F32)
    step(f"FP8Experts with choices outside the experts, {ids_dtype}")
    poison = torch.full((1 << 20,), float("nan"), device="cuda")   # so that memory handed out next holds NaN
    del poison
    xd, idd, wd = dev(x).view(2, 3, k), dev(ids).to(ids_dtype).view(2, 3, 2), dev(weights).view(2, 3, 2)
    y = m(xd, idd, wd)
    clean = np.where((ids >= 0) & (ids < e), weights, 0)
    ref, tol = _experts_reference(x, w1, w2, ids, clean, F32)
    assert y.shape == (2, 3, k) and (np.abs(host(y.double()).reshape(6, k) - ref) <= tol).all()
    assert (host(y)[0, 1] == 0).all()
    if ids_dtype == torch.int64:
        far = idd.clone()
        far[far == 4] = 1 << 32       # not expert 0
        far[far == 200] = -(1 << 40) + 1
        assert torch.equal(m(xd, far, wd), y)
    assert m(xd[:0], idd[:0], wd[:0]).shape == (0, 3, k)


def test_experts_do_not_depend_on_the_batch():
    """A token's output has the same bits alone and beside others with the same number of rows of every expert's form."""
    rng = np.random.default_rng(9)
    m, _, _ = _experts(rng, 8, 256, 128, BF16)
    x, ids = dev(_x(rng, 64, 256)).to(BF16), torch.randint(0, 8, (64, 2), device="cuda")
    w = torch.rand(64, 2, device="cuda")
    step("FP8Experts, tokens in another order")
    y = m(x, ids, w)
    p = torch.randperm(64, device="cuda")
    assert torch.equal(m(x[p], ids[p], w[p]), y[p])
    assert torch.equal(m(x, ids, w), y)


def test_router_and_experts_together_with_gradients():
    """Logits to outputs, and the gradient of a loss with respect to the logits by the formula."""
    rng = np.random.default_rng(11)
    t, e, top, k, inner = 40, 12, 3, 128, 64
    m, w1, w2 = _experts(rng, e, k, inner, F32)
    x = dev(_x(rng, t, k))
    logits = dev(rng.standard_normal((t, e)).astype(np.float32)).requires_grad_()
    dy = dev(rng.standard_normal((t, k)).astype(np.float32))
    step("router, experts and their gradient")
    how = dict(score="sigmoid", groups=4, top_groups=2, scale=1.5)
    ids, w = L().route(logits, top, bias=torch.zeros(e, device="cuda"), **how)
    y = m(x, ids, w)
    y.backward(dy)
    hi, hw = host(ids), host(w.detach())
    ref, tol = _experts_reference(host(x), w1, w2, hi, hw, F32)
    assert (np.abs(host(y.detach().double()) - ref) <= tol).all()
    # dL/dw_j = dy . (expert j's output), from outputs with one weight each
    dw, dtol = np.zeros((t, top)), np.zeros((t, top))
    for j in range(top):
        one = np.zeros((t, top), np.float32)
        one[:, j] = 1
        part, off = _experts_reference(host(x), w1, w2, hi, one, F32)
        d = np.abs(host(dy).astype(np.float64))
        dw[:, j] = (part * host(dy)).sum(1)
        dtol[:, j] = (d * (off + k * 2.0 ** -23 * np.abs(part))).sum(1)
    ref = OM.route_backward(host(logits.detach()), hi, dw, score="sigmoid", scale=1.5)
    # (a weight's derivative by a logit is at most scale / 4 here, by every choice of the token)
    tol = 1.5 * dtol.sum(1, keepdims=True) + 2.0 ** -22 * 1.5 * np.abs(dw).sum(1, keepdims=True)
    assert (np.abs(host(logits.grad.double()) - ref) <= tol).all()


def test_gradients_that_are_not_computed_are_refused():
    rng = np.random.default_rng(2)
    m, _, _ = _experts(rng, 4, 64, 32, F32)
    lin = L().FP8Linear.from_weight(torch.randn(64, 64, device="cuda"), torch.ones(64, device="cuda"))
    x, ids, w = torch.randn(5, 64, device="cuda"), torch.randint(0, 4, (5, 2), device="cuda"), torch.rand(5, 2, device="cuda")
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    step("FP8 modules refuse their input's gradient")
    plain = lin(x)
    y = lin(xg)
    assert not plain.requires_grad and torch.equal(y, plain)
    y += 1
    for loss in (y, xg + lin(xg)):
        with pytest.raises(RuntimeError, match="FP8Linear has no backward pass"):
            loss.sum().backward()
    plain = m(x, ids, w)
    assert not plain.requires_grad
    for weights in (w, wg):
        for residual in (False, True):
            y = m(xg, ids, weights)
            assert torch.equal(y, plain)
            with pytest.raises(RuntimeError, match="FP8Experts has no backward pass"):
                (xg + y if residual else y).sum().backward()
    with torch.no_grad():
        assert not m(xg, ids, wg).requires_grad
    with torch.inference_mode():
        assert torch.equal(m(x, ids, w), plain) and torch.equal(lin(x), lin(x.clone()))
    for dtype in (torch.float64, torch.float16):
        wd = w.to(dtype).requires_grad_()
        m(x, ids, wd).sum().backward()
        assert wd.grad.dtype == dtype


@pytest.mark.parametrize("t", [1, 16, 300, 3000])
def test_route_and_experts_captured_and_replayed(t):
    rng = np.random.default_rng(t)
    m, _, _ = _experts(rng, 16, 128, 64, BF16)
    x = dev(_x(rng, t, 128)).to(BF16)
    logits = torch.randn(t, 16, device="cuda")
    step(f"route and FP8Experts captured, {t} tokens")

    def call():
        return m(x, *L().route(logits, 6, score="sigmoid", groups=4, top_groups=2))

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = call()
    for i in range(3):
        logits.normal_()
        logits[:, i] = float("-inf")
        x.copy_(dev(_x(rng, t, 128)))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, call())


def test_two_streams_at_once():
    rng = np.random.default_rng(6)
    m, _, _ = _experts(rng, 8, 256, 128, BF16)
    calls = [(dev(_x(rng, n, 256)).to(BF16), torch.randint(0, 8, (n, 4), device="cuda"), torch.rand(n, 4, device="cuda")) for n in (3000, 40)]
    step("FP8Experts on two streams")
    ref = [m(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(m(*c))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, ref[i % 2])
