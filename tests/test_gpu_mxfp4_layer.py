"""MXFP4 modules on the GPU: quantising, products and products grouped by expert run together.

First products have integer activations and weights whose sums fit 24 bits, so the gate and up values are exact
and the inner activations (silu and the rounding of the second product's input) can be formed from the oracle's
values by the same elementwise call.  The second product then differs from its 64-bit value by at most I 2^-23 of
the sum of the magnitudes, and the sum over a token's choices by 2^-23 a choice of theirs.
"""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as O
from tests.gpu_util import dev, host, step

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def L():
    from weight_only_bit_group_amd import layer
    return layer


def _ints(rng, *shape):
    """Values that MXFP4 holds exactly with the factor 1: every block has a 4 or a 6."""
    v = rng.choice(np.array([0, .5, 1, 1.5, 2, 3, 4, 6]), shape) * rng.choice([-1.0, 1.0], shape)
    v[..., ::32] = rng.choice([4.0, -6.0], v[..., ::32].shape)
    return v.astype(np.float32)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 256), (2, 3, 96), (40, 256), (300, 2080)])
def test_linear_of_integers_is_exact(shape, dtype, act):
    rng = np.random.default_rng(shape[-1] + len(shape))
    k, n = shape[-1], 67
    w, x, b = _ints(rng, n, k), _ints(rng, *shape), rng.integers(-9, 9, n).astype(np.float32)
    step(f"MXFP4Linear {shape} {dtype} {act}")
    lin = L().MXFP4Linear.from_weight(dev(w), dev(b), act)
    y = lin(dev(x).to(dtype))
    assert y.dtype == F32 and tuple(y.shape) == (*shape[:-1], n)
    assert (host(y) == x.astype(np.float64) @ w.T.astype(np.float64) + b).all()
    state = {name: t.clone() for name, t in lin.state_dict().items()}
    other = L().MXFP4Linear(torch.zeros_like(lin.codes), torch.zeros_like(lin.scales), torch.zeros_like(lin.bias), act)
    other.load_state_dict(state)
    assert torch.equal(other(dev(x).to(dtype)), y)


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_linear_takes_rows_of_any_layout(act):
    """Transposed, sliced at odd elements, broadcast and empty inputs equal the dense ones."""
    rng = np.random.default_rng(5)
    lin = L().MXFP4Linear.from_weight(dev(_ints(rng, 40, 64)), None, act)
    base = dev(_ints(rng, 9, 130)).to(BF16)
    step(f"MXFP4Linear over views, {act}")
    for x in (base[:, 3:67], base[:, 8:72], base[1:, :64], base[:1, :64].expand(7, 64),
              dev(_ints(rng, 64, 12)).to(BF16).t(), base.reshape(-1)[1:65], base[:0, :64]):
        assert torch.equal(lin(x), lin(x.clone(memory_format=torch.contiguous_format)))
    assert lin(base[:0, :64]).shape == (0, 40)


def _experts_reference(x, w1, w2, ids, weights, act):
    """(values, sums of magnitudes) of the experts in 64 bits; x, w1 exact."""
    t, top = ids.shape
    inner, k = w2.shape[2], w2.shape[1]
    y, mag = np.zeros((t, k)), np.zeros((t, k))
    for j in range(top):
        for i in range(t):
            e = int(ids[i, j])
            if not 0 <= e < len(w1):
                continue
            g = dev((w1[e].astype(np.float64) @ x[i].astype(np.float64)).astype(np.float32)[None])
            h = torch.nn.functional.silu(g[:, :inner]) * g[:, inner:]
            if act == "bf16":
                h = host(h.to(BF16).double())[0]
            else:
                h = O.dequantize(*O.quantize(host(h)))[0]
            y[i] += float(weights[i, j]) * (w2[e].astype(np.float64) @ h)
            mag[i] += abs(float(weights[i, j])) * (np.abs(w2[e]).astype(np.float64) @ np.abs(h))
    return y, mag


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("t,top,e,k,inner", [(1, 2, 4, 64, 32), (1, 8, 16, 256, 96), (5, 1, 3, 96, 64),
                                             (33, 2, 5, 64, 160), (150, 4, 7, 128, 64)])
def test_experts(t, top, e, k, inner, act):
    rng = np.random.default_rng(t * 100 + e)
    w1, w2 = _ints(rng, e, 2 * inner, k), _ints(rng, e, k, inner)
    x = _ints(rng, t, k)
    ids = np.stack([rng.permutation(e)[:top] for _ in range(t)]) if top <= e else rng.integers(0, e, (t, top))
    weights = rng.random((t, top)).astype(np.float32)
    step(f"MXFP4Experts t {t} top {top} e {e} k {k} inner {inner} {act}")
    m = L().MXFP4Experts.from_weights(dev(w1), dev(w2), act)
    y = m(dev(x).to(BF16), dev(ids), dev(weights))
    ref, mag = _experts_reference(x, w1, w2, ids, weights, act)
    assert y.dtype == F32
    err = np.abs(host(y).astype(np.float64) - ref)
    assert (err <= (inner + 2 * top) * 2.0 ** -23 * mag).all(), (err / (mag + 1e-300)).max()


@pytest.mark.parametrize("ids_dtype", [torch.int64, torch.int32, torch.uint8])
def test_experts_with_choices_that_add_nothing(ids_dtype):
    """Choices outside the range, tokens without a valid one, an expert chosen twice by a token, and no tokens."""
    rng = np.random.default_rng(3)
    e, k, inner = 4, 64, 32
    w1, w2, x = _ints(rng, e, 2 * inner, k), _ints(rng, e, k, inner), _ints(rng, 6, k)
    ids = np.array([[0, 1], [4, 4], [200, 2], [3, 3], [1, 99], [4, 0]])
    weights = rng.random((6, 2)).astype(np.float32)
    weights[(ids < 0) | (ids >= e)] = np.nan
    m = L().MXFP4Experts.from_weights(dev(w1), dev(w2))
    step(f"MXFP4Experts with choices outside the experts, {ids_dtype}")
    poison = torch.full((1 << 20,), float("nan"), device="cuda")   # so that memory handed out next holds NaN
    del poison
    xd, idd, wd = dev(x).view(2, 3, k), dev(ids).to(ids_dtype).view(2, 3, 2), dev(weights).view(2, 3, 2)
    y = m(xd, idd, wd)
    assert tuple(y.shape) == (2, 3, k)
    ref, mag = _experts_reference(x, w1, w2, ids, weights, "bf16")
    assert (np.abs(host(y).reshape(6, k).astype(np.float64) - ref) <= (inner + 4) * 2.0 ** -23 * mag).all()
    assert (host(y).reshape(6, k)[1] == 0).all()
    if ids_dtype is not torch.uint8:
        none = m(xd, torch.full_like(idd, -1), wd)
        assert (host(none) == 0).all()
    assert m(xd[:0], idd[:0], wd[:0]).shape == (0, 3, k)


def test_experts_do_not_depend_on_the_batch_order():
    """Tokens permuted: the same sums of each token, bit for bit (its products are added in its own order)."""
    rng = np.random.default_rng(9)
    e, k, inner, t, top = 8, 128, 64, 64, 4
    m = L().MXFP4Experts.from_weights(dev(rng.standard_normal((e, 2 * inner, k)).astype(np.float32)),
                                      dev(rng.standard_normal((e, k, inner)).astype(np.float32)))
    x = dev(rng.standard_normal((t, k)).astype(np.float32))
    ids, weights = dev(rng.integers(0, e, (t, top))), dev(rng.random((t, top)).astype(np.float32))
    perm = dev(rng.permutation(t))
    step("MXFP4Experts over permuted tokens")
    assert torch.equal(m(x, ids, weights)[perm], m(x[perm], ids[perm], weights[perm]))


def test_modules_refuse():
    m = L().MXFP4Experts.from_weights(torch.zeros(2, 64, 64, device="cuda"), torch.zeros(2, 64, 32, device="cuda"))
    x, ids, w = torch.zeros(3, 64, device="cuda"), torch.zeros(3, 2, dtype=torch.int64, device="cuda"), \
        torch.zeros(3, 2, device="cuda")
    for bad in ((x[:, :32], ids, w), (x, ids[:2], w), (x, ids, w[:, :1]), (x, ids.float(), w), (x, ids[:, :0], w[:, :0]),
                (x, ids.bool(), w)):
        with pytest.raises(ValueError):
            m(*bad)
    lin = L().MXFP4Linear.from_weight(torch.zeros(8, 64, device="cuda"))
    with pytest.raises(ValueError):
        lin(x[:, :32])
    with pytest.raises(ValueError):
        L().MXFP4Linear.from_weight(torch.zeros(8, 48, device="cuda"))
    with pytest.raises(ValueError, match="already quantized"):
        L().plan_quantization(torch.nn.ModuleDict({"q": lin, "k": torch.nn.Linear(32, 32)}), ("q",))


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_gradients_are_the_formulas_or_refused(act):
    """Inputs that require a gradient: the same outputs, the router's weights' gradient, and an error for the rest."""
    rng = np.random.default_rng(12)
    e, k, inner, t, top = 5, 64, 32, 6, 2
    lin = L().MXFP4Linear.from_weight(dev(_ints(rng, 40, k)), None, act)
    m = L().MXFP4Experts.from_weights(dev(_ints(rng, e, 2 * inner, k)), dev(_ints(rng, e, k, inner)), act)
    x, w = dev(_ints(rng, t, k)), dev(rng.random((t, top)).astype(np.float32))
    ids = dev(np.stack([rng.permutation(e)[:top] for _ in range(t)]))
    step(f"MXFP4 modules with inputs that require a gradient, {act}")
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    assert torch.equal(lin(xg), lin(x)) and torch.equal(m(xg, ids, wg), m(x, ids, w))
    for y in (lin(xg), m(xg, ids, w), xg + m(xg, ids, wg)):
        with pytest.raises(RuntimeError, match="has no backward pass"):
            y.sum().backward()
    dy = dev(rng.integers(-3, 4, (t, k)).astype(np.float32))
    wg = w.clone().requires_grad_()   # (the refused passes may have reached the other)
    m(x, ids, wg).backward(dy)
    for j in range(top):
        one = torch.zeros_like(w)
        one[:, j] = 1
        part = (m(x, ids, one) * dy).double()
        # k products and sums in fp32, each off by half a step of the magnitudes at most
        assert ((wg.grad[:, j] - part.sum(1)).abs() <= (k + 1) * 2.0 ** -24 * part.abs().sum(1)).all()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("t,top", [(1, 8), (64, 8), (600, 8), (4096, 4), (1 << 17, 8)])
def test_experts_captured_and_replayed(t, top, act):
    """A captured call follows its inputs over several replays, with the program's own calls between them."""
    rng = np.random.default_rng(t + top)
    e, k, inner = 16, 64, 32
    m = L().MXFP4Experts.from_weights(dev(_ints(rng, e, 2 * inner, k)), dev(_ints(rng, e, k, inner)), act)

    def inputs():
        ids = rng.integers(0, e + 1, (t, top))   # (choice e adds nothing)
        return dev(rng.standard_normal((t, k)).astype(np.float32)).to(BF16), dev(ids), dev(rng.random((t, top)).astype(np.float32))

    held = inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m(*held)
    for i in range(5):
        step(f"MXFP4Experts {act}, {t} tokens of {top} choices, replay {i}")
        new = inputs()
        want = m(*new)
        for old, value in zip(held, new):
            old.copy_(value)
        torch.cuda.synchronize()
        graph.replay()
        again = m(*new)
        assert torch.equal(y, want) and torch.equal(again, want)
