"""Routing, its gradient, the choices grouped by expert, the gated activation and the weighted sum on the GPU against
the 64-bit oracle.

Routing is formed in 64 bits and rounded once, so choices are equal and weights within 2^-24 of the value (and the
64-bit arithmetic's own 2^-45, taken generously: some hundred roundings).  Sums of n products in fp32 are off by at most
n 2^-23 of the sum of their magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import fp8 as O8
from oracle import moe as O
from tests.gpu_util import dev, host, step

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def B():
    from weight_only_bit_group_amd import binding
    return binding


def L():
    from weight_only_bit_group_amd import layer
    return layer


HALF = 2.0 ** -24 + 2.0 ** -45


def _same(got, ref, what):
    ids, w = host(got[0]), host(got[1].double())
    assert got[0].dtype == torch.int32 and got[1].dtype == F32
    assert (ids == ref[0]).all(), (what, np.argwhere((ids != ref[0]).any(1))[:3])
    assert (np.isnan(w) == np.isnan(ref[1])).all()
    assert (np.abs(np.nan_to_num(w) - np.nan_to_num(ref[1])) <= HALF * np.abs(np.nan_to_num(ref[1])) + 2.0 ** -149).all(), what


ROUTES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (7, 64, 8, 1, 1), (33, 60, 6, 4, 2), (16, 256, 8, 8, 4), (50, 100, 10, 1, 1), (9, 130, 5, 13, 3),
          (40, 384, 8, 1, 1), (5, 512, 20, 64, 7), (12, 1000, 64, 1, 1), (6, 1024, 16, 32, 5), (300, 128, 8, 2, 1), (20, 21, 3, 7, 7)]


@pytest.mark.parametrize("t,e,top,groups,top_groups", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route(t, e, top, groups, top_groups, score, dtype):
    rng = np.random.default_rng(t * 31 + e)
    l = rng.standard_normal((t, e)) * 3
    l[rng.random((t, e)) < 0.15] = -INF
    if t > 4:
        l[3] = -INF
        l[2, :] = 1.25           # all equal: the lowest indices
    x = dev(l.astype(np.float32)).to(dtype)
    l = host(x.double())
    bias = (rng.standard_normal(e) * 0.2).astype(np.float32)
    step(f"route {t} x {e} top {top} groups {top_groups} of {groups} {score} {dtype}")
    for b in (None, bias):
        for renormalize in (True, False):
            how = dict(score=score, groups=groups, top_groups=top_groups, renormalize=renormalize, scale=2.5)
            got = B().aq_moe_route(x, top, bias=None if b is None else dev(b), **how)
            _same(got, O.route(l, top, bias=b, **how), (b is not None, renormalize))


def test_route_of_ties_and_near_ties():
    """Keys equal in 64 bits go to the lowest index; keys that differ below a 32-bit rounding are told apart."""
    rng = np.random.default_rng(5)
    l = rng.choice([0.5, 1.0, -2.0], (200, 192)).astype(np.float32)
    step("route ties")
    for score in ("softmax", "sigmoid"):
        for bias in (None, np.zeros(192, np.float32), rng.choice([0.0, 0.25], 192).astype(np.float32)):
            for groups, tg in ((1, 1), (8, 3)):
                how = dict(score=score, groups=groups, top_groups=tg)
                _same(B().aq_moe_route(dev(l), 12, bias=None if bias is None else dev(bias), **how), O.route(l, 12, bias=bias, **how), score)
    base = np.full((300, 128), 3.0, np.float32)
    near = (base + rng.integers(-4, 5, base.shape) * 2.0 ** -22).astype(np.float32)
    for bias in (None, (rng.integers(-3, 4, 128) * 2.0 ** -26).astype(np.float32)):
        how = dict(score="sigmoid", renormalize=False)
        _same(B().aq_moe_route(dev(near), 9, bias=None if bias is None else dev(bias), **how), O.route(near, 9, bias=bias, **how), "near")


def test_route_of_masks_infinities_and_nan():
    low = float(np.finfo(np.float32).min)
    l = np.array([[1, 2, 3, 4], [-INF, 2, -INF, 4], [-INF] * 4, [low] * 4, [low, low, -INF, 1], [np.nan, 1, 2, 3], [INF, 1, 2, 3],
                  [-INF, np.nan, -INF, -INF], [1e30, -1e30, 0, 0], [-800, -900, -1000, -1e5], [-0.0, 0.0, -0.0, 0.0]], np.float32)
    l = np.concatenate([l, l[:, ::-1], np.full((11, 4), -INF, np.float32)], 1)
    step("route masks, infinities, NaN")
    bias = np.array([0.1] * 12, np.float32)
    for b in (None, bias, np.where(np.arange(12) == 1, -np.float32(INF), bias), np.where(np.arange(12) == 4, np.float32(INF), bias)):
        for score in ("softmax", "sigmoid"):
            for renormalize in (True, False):
                for groups, tg in ((1, 1), (3, 2), (3, 1)):
                    how = dict(score=score, renormalize=renormalize, groups=groups, top_groups=tg)
                    _same(B().aq_moe_route(dev(l), 3, bias=None if b is None else dev(b), **how), O.route(l, 3, bias=b, **how), how)
    bad = bias.copy()
    bad[7] = np.nan
    ids, w = B().aq_moe_route(dev(l), 3, bias=dev(bad))
    assert (host(ids) == [0, 1, 2]).all() and w.isnan().all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("t,e,top", [(1, 4, 1), (9, 64, 8), (37, 100, 6), (20, 256, 8), (6, 1000, 33)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_gradient(t, e, top, score, renormalize, dtype):
    rng = np.random.default_rng(t + e)
    l = rng.standard_normal((t, e)) * 2
    l[rng.random((t, e)) < 0.2] = -INF
    if t > 3:
        l[2] = -INF
    x = dev(l.astype(np.float32)).to(dtype).requires_grad_()
    d = rng.standard_normal((t, top)).astype(np.float32)
    how = dict(score=score, renormalize=renormalize, scale=2.5)
    step(f"route gradient {t} x {e} top {top} {score} renormalize {renormalize} {dtype}")
    ids, w = L().route(x, top, **how)
    assert w.requires_grad and not ids.requires_grad
    w.backward(dev(d))
    l = host(x.detach().double())
    ref = O.route_backward(l, host(ids), d, **how)
    got = host(x.grad.double())
    assert x.grad.dtype == dtype
    # 64-bit sums of terms that cancel (2^-45 of the largest), then one rounding
    tol = 2.0 ** -45 * 2.5 * np.abs(d).max(1, keepdims=True) * (top + 1) + (2.0 ** -24 if dtype == F32 else 2.0 ** -8) * np.abs(ref)
    assert (np.abs(got - ref) <= tol).all()
    # the same against differences of the weights themselves, in the direction of the gradient's own entries
    again = torch.autograd.grad(L().route(x, top, **how)[1], x, dev(d))[0]
    assert torch.equal(again, x.grad)


def test_route_gradient_of_a_token_without_finite_weights():
    l = torch.tensor([[1.0, float("nan"), 0.0, 2.0], [1.0, 2.0, 3.0, 4.0]], device="cuda", requires_grad=True)
    step("route gradient of NaN")
    ids, w = L().route(l, 2)
    w.sum().backward()
    assert l.grad[0, :2].isnan().all() and (l.grad[1].abs() < 1e-6).all()


def test_route_takes_leading_dimensions_strides_and_other_types():
    rng = np.random.default_rng(1)
    wide = dev(rng.standard_normal((24, 80)).astype(np.float32))
    step("route of views")
    ref = B().aq_moe_route(wide[:, 8:72].contiguous(), 4)
    for x in (wide[:, 8:72], wide[:, 8:72].reshape(2, 3, 4, 64), wide.t()[8:72].t(), wide[:, 8:72].double().float()):
        ids, w = L().route(x, 4)
        assert ids.shape == w.shape == (*x.shape[:-1], 4)
        assert torch.equal(ids.view(-1, 4), ref[0]) and torch.equal(w.view(-1, 4), ref[1])
    half = wide[:, 8:72].half()
    assert torch.equal(L().route(half, 4)[0], L().route(half.float(), 4)[0])
    h = half.clone().requires_grad_()
    L().route(h, 4)[1][:, 0].sum().backward()
    assert h.grad.dtype == torch.float16 and h.grad.isfinite().all()
    assert L().route(wide[:0], 4)[0].shape == (0, 4) and L().route(wide[:1, :1], 1)[1].item() == 1.0
    for bad in (dict(top=0), dict(top=81), dict(top=4, groups=3), dict(top=4, groups=8, top_groups=9), dict(top=4, score="relu"),
                dict(top=4, bias=wide[0, :5]), dict(top=4, scale=float("inf")), dict(top=11, groups=8, top_groups=1)):
        with pytest.raises(ValueError):
            L().route(wide, **bad)


# ---- grouped by expert -------------------------------------------------------------------------------

GROUPS = [(0, 2, 4), (1, 1, 1), (1, 8, 64), (3, 2, 5), (64, 8, 128), (1000, 4, 32), (700, 6, 1024), (2048, 8, 60), (4096, 4, 513),
          (2049, 8, 7), (5000, 8, 256), (16384, 8, 128), (20011, 3, 1000)]


@pytest.mark.parametrize("t,top,e", GROUPS)
def test_group(t, top, e):
    rng = np.random.default_rng(t + e)
    ids = rng.integers(-2, e + 2, (t, top)).astype(np.int32)
    ids[rng.random((t, top)) < 0.3] = e // 2          # one expert far more popular
    if t > 2:
        ids[1] = rng.choice([-2 ** 31, 2 ** 31 - 1, e, -1], top)
    step(f"group {t} x {top} over {e}")
    off, rows, slots = (host(v) for v in B().aq_moe_group(dev(ids), e))
    ref = O.group(ids, e)
    assert (off == ref[0]).all() and (rows[:off[-1]] == ref[1]).all() and (slots == ref[2]).all()
    assert rows.shape == (t * top,)


def test_group_of_one_expert_and_of_none():
    step("group of one expert and of none")
    for c in (100, 30000):
        off, rows, slots = B().aq_moe_group(torch.full((c, 1), 3, dtype=torch.int32, device="cuda"), 8)
        assert host(off).tolist() == [0, 0, 0, 0] + [c] * 5 and torch.equal(rows, torch.arange(c, device="cuda", dtype=torch.int32))
        assert torch.equal(slots[:, 0], rows)
        off, rows, slots = B().aq_moe_group(torch.full((c, 1), -1, dtype=torch.int32, device="cuda"), 8)
        assert (off == 0).all() and (slots == -1).all()


def test_group_captured_with_a_workspace_of_its_own():
    ids = torch.randint(0, 64, (6000, 8), dtype=torch.int32, device="cuda")
    ws = torch.empty(B().aq_moe_group_workspace(6000, 8, 64), dtype=torch.uint8, device="cuda")
    step("group captured and replayed")
    B().aq_moe_group(ids, 64, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = B().aq_moe_group(ids, 64, ws)
    for _ in range(3):
        ids.random_(-1, 65)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, B().aq_moe_group(ids, 64)):
            n = int(got[0][-1]) if a.dim() == 1 and a.shape[0] > 65 else None
            assert torch.equal(a[:n], b[:n])
    with pytest.raises(ValueError, match="workspace"):
        B().aq_moe_group(ids, 64, ws[:64])
    with pytest.raises(ValueError):
        B().aq_moe_group(ids, 1025)
    with pytest.raises(ValueError):
        B().aq_moe_group(ids.long(), 64)


# ---- between and behind the products -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,inner", [(1, 16), (5, 144), (40, 1408), (300, 272)])
def test_swiglu_quantize(m, inner, dtype):
    """The gated values differ from their 64-bit values by some 2^-20; the rounding to FP8 of a value that close to the
    middle between two codes may take either, every other code is the oracle's."""
    rng = np.random.default_rng(m + inner)
    h = dev((rng.standard_normal((m, 2 * inner)) * 3).astype(np.float32)).to(dtype)
    step(f"swiglu quantize {m} x {inner} {dtype}")
    c, s = B().aq_fp8_swiglu_quantize(h)
    v = host(h.double())
    g, u = v[:, :inner], v[:, inner:]
    ref = g / (1 + np.exp(-g)) * u
    # exp2 of -g log2 e: its argument's rounding, |g| 2^-24 log2 e twice, and three operations within 2^-23
    rel = (2 * np.abs(g) + 8) * 2.0 ** -23
    s = host(s).astype(np.float64)
    top = np.maximum.reduceat(np.abs(ref), np.arange(0, inner, 128), axis=1)
    assert (np.abs(s * 448 - top) <= (rel.max() + 2.0 ** -22) * top).all()
    y = O8.decode(host(c.view(torch.uint8)))
    q = ref / np.repeat(s, 128, 1)[:, :inner]
    lo, hi = (O8.decode(O8.encode(np.clip(q * (1 + f * (rel + 2.0 ** -22)), -448, 448))) for f in (-1, 1))
    assert ((y == lo) | (y == hi)).all()
    assert (lo != hi).mean() < 1e-3


def test_swiglu_quantize_leaves_rows_behind_the_end():
    h = torch.randn(50, 320, device="cuda")
    codes, scales = torch.full((50, 160), 9, dtype=torch.uint8, device="cuda"), torch.full((50, 2), 9.0, device="cuda")
    ref = B().aq_fp8_swiglu_quantize(h)
    h[20:] = float("nan")
    step("swiglu quantize to an end")
    for end in (20, 0, 50, 99, -3):
        codes.fill_(9), scales.fill_(9)
        B().aq_fp8_swiglu_quantize(h, torch.tensor([end], dtype=torch.int32, device="cuda"), codes=codes, scales=scales)
        n = min(max(end, 0), 50)
        m = min(n, 20)
        assert torch.equal(codes[:m], ref[0].view(torch.uint8)[:m]) and torch.equal(scales[:m], ref[1][:m])
        assert scales[20:n].isnan().all() and (codes[20:n] == 0).all()
        assert (codes[n:] == 9).all() and (scales[n:] == 9).all()
    for bad in (h[:, :300], h[:, :16], h.half(), h[:, ::2], h[None]):
        with pytest.raises(ValueError):
            B().aq_fp8_swiglu_quantize(bad)


@pytest.mark.parametrize("ydt,odt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("t,top,k,r", [(1, 1, 8, 1), (3, 8, 64, 9), (50, 2, 2048, 100), (33, 64, 136, 500), (400, 6, 1000, 37)])
def test_combine_and_its_gradient(t, top, k, r, ydt, odt):
    rng = np.random.default_rng(t + k)
    y = dev(rng.standard_normal((r, k)).astype(np.float32)).to(ydt)
    slots = rng.integers(-1, r + 1, (t, top)).astype(np.int32)
    slots[0, 0] = 2 ** 31 - 1
    w = rng.standard_normal((t, top)).astype(np.float32)
    inside = (slots >= 0) & (slots < r)
    w[~inside] = np.nan
    step(f"combine {t} x {top} x {k} {ydt} {odt}")
    out = B().aq_moe_combine(y, dev(slots), dev(w), odt)
    rows = np.where(inside[..., None], host(y.double())[np.where(inside, slots, 0)], 0.0)
    parts = rows * np.where(inside, w, 0.0).astype(np.float64)[..., None]
    tol = top * 2.0 ** -23 * np.abs(parts).sum(1)
    ref = parts.sum(1)
    if odt == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert out.dtype == odt and (np.abs(host(out.double()) - ref) <= tol).all()
    d = dev(rng.standard_normal((t, k)).astype(np.float32)).to(odt)
    dw = B().aq_moe_combine_backward(y, dev(slots), d)
    prod = rows * host(d.double())[:, None]
    assert dw.dtype == F32 and (np.abs(host(dw.double()) - prod.sum(2)) <= k * 2.0 ** -23 * np.abs(prod).sum(2)).all()
    assert (host(dw)[~inside] == 0).all()


def test_combine_refusals():
    y, slots, w = torch.randn(5, 64, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda")
    step("combine refusals")
    for bad in ((y.half(), slots, w), (y[:, :60].contiguous(), slots, w), (y, slots.long(), w), (y, slots, w.double()), (y, slots, w[:, :1]),
                (y.t(), slots, w), (y[:0], slots, w), (y, slots, w, torch.float16)):
        with pytest.raises(ValueError):
            B().aq_moe_combine(*bad)
    assert B().aq_moe_combine(y, slots[:0], w[:0]).shape == (0, 64)
    out = torch.empty(3, 64, dtype=BF16, device="cuda")
    assert B().aq_moe_combine(y, slots, w, out=out) is out
