"""What route's derivatives are and which are refused; one token's logits in any layout."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fw

from oracle import moe as O
from tests.gpu_util import dev, host, step
from tests.test_gpu_route_graph import HOWS, _gpu, _logits, route  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("groups,top_groups,bias", [(1, 1, False), (1, 1, True), (4, 2, False), (4, 2, True), (8, 8, True)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_against_differences_in_64_bits(route, dtype, groups, top_groups, bias, renormalize, score):
    """(f(l + h) - f(l - h)) / 2h of f = sum_j d_j w_j at the choices that were made, formed in 64 bits.  A weight as a
    function of one logit has a third derivative below 2 scale (a logistic function's is below 1/8), so the difference is
    off by h^2 / 3 scale sum |d|, and by the 64-bit weights' roundings over h; the gradient by its one rounding."""
    t, e, top, scale, h = 7, 40, 5, 2.5, 2.0 ** -12
    rng = np.random.default_rng(e + groups)
    l = rng.standard_normal((t, e)) * 2
    l[rng.random((t, e)) < 0.2] = -np.inf
    l[3] = -np.inf          # nothing to choose
    l[4, 2:] = -np.inf      # fewer than top
    b = (rng.standard_normal(e) * 0.2).astype(np.float32) if bias else None
    d = rng.standard_normal((t, top)).astype(np.float32)
    x = dev(l.astype(np.float32)).to(dtype).requires_grad_()
    l = host(x.detach().double())
    kept = dict(score=score, renormalize=renormalize, scale=scale)
    step(f"route against differences, {score} renormalize {renormalize} groups {groups} bias {bias} {dtype}")
    ids, w = route(x, top, bias=None if b is None else dev(b), groups=groups, top_groups=top_groups, **kept)
    assert (host(ids) == O.route(l, top, bias=b, groups=groups, top_groups=top_groups, **kept)[0]).all()
    got, = torch.autograd.grad(w, x, dev(d))
    got, ids = host(got.double()), host(ids)
    diff = np.zeros((t, e))
    for i in range(e):
        side = []
        for s in (h, -h):
            moved = l.copy()
            moved[:, i] += s
            side.append((O.weights_at(moved, ids, **kept) * d).sum(1))
        diff[:, i] = (side[0] - side[1]) / (2 * h)
    size = scale * np.abs(d).sum(1, keepdims=True)
    tol = size * (h * h / 3 * 2 + 2.0 ** -48 / h) + (2.0 ** -24 if dtype == F32 else 2.0 ** -8) * np.abs(diff) * 1.01
    assert (np.abs(got - diff) <= tol).all()
    assert (got[3] == 0).all() and np.abs(got).max() > 1e-3
    assert (np.abs(got - O.route_backward(l, ids, d, **kept)) <= size * 2.0 ** -45 * (top + 1) + (2.0 ** -24 if dtype == F32 else 2.0 ** -8) * np.abs(got) * 1.01).all()


@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("needs", [True, False])
def test_derivative_of_the_gradient_is_refused(route, how, needs):
    """The gradient is a function of the logits whatever the gradient that comes in: with create_graph, asking for its
    derivative is an error, never nothing."""
    l = _logits().requires_grad_()
    d = torch.randn(9, 3, device="cuda", requires_grad=needs)
    step(f"route's second derivative, {how}")
    plain, = torch.autograd.grad(route(l, 3, **how)[1], l, d)
    assert not plain.requires_grad
    _, w = route(l, 3, **how)
    g, = torch.autograd.grad(w, l, d, create_graph=True)
    assert torch.equal(g, plain)
    with pytest.raises(RuntimeError, match="differentiate"):
        torch.autograd.grad(g.square().sum(), l)
    _, w = route(2 * l, 3, **how)
    penalty = torch.autograd.grad(w.sum(), l, create_graph=True)[0].square().sum()
    with pytest.raises(RuntimeError, match="differentiate"):
        (w.square().sum() + penalty).backward()
    other = _logits(seed=1).requires_grad_()
    _, w = route(other, 3, **how)
    w.square().sum().backward(create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate"):
        other.grad.sum().backward()
    other.grad = None


def test_forward_derivatives_are_refused(route):
    from weight_only_bit_group_amd import layer
    l = _logits()
    t = torch.randn_like(l)
    ref = route(l, 3)
    step("route of logits with a tangent")
    with fw.dual_level():
        for dual in (fw.make_dual(l, t), fw.make_dual(l.clone().requires_grad_(), t), fw.make_dual(l.double(), t.double()),
                     fw.make_dual(l.view(3, 3, 24), t.view(3, 3, 24)), fw.make_dual(l, t) * 2.0):
            with pytest.raises(RuntimeError, match="forward"):
                route(dual, 3)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward"):
                route(dual, 3)
        got = route(l, 3)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        got = route(fw.unpack_dual(fw.make_dual(l, t)).primal, 3)
        assert torch.equal(got[1], ref[1])
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: route(x, 3)[1], (l,), (t,))
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: route(x, 3)[1].sum())(l)

    lin = layer.FP8Linear.from_weight(torch.randn(48, 64, device="cuda"))
    m = layer.FP8Experts.from_weights(torch.randn(4, 64, 32, device="cuda"), torch.randn(4, 32, 32, device="cuda"))
    x, ids, w = torch.randn(9, 32, device="cuda"), torch.randint(0, 4, (9, 2), device="cuda"), torch.rand(9, 2, device="cuda")
    v = torch.randn(9, 64, device="cuda")
    step("FP8 modules of inputs with a tangent")
    with fw.dual_level():
        for call in (lambda: lin(fw.make_dual(v, v)), lambda: lin(fw.make_dual(v.half(), v.half())), lambda: m(fw.make_dual(x, x), ids, w),
                     lambda: m(x, ids, fw.make_dual(w, w)), lambda: m(x, ids, fw.make_dual(w.double(), w.double())),
                     lambda: m(x, ids, fw.make_dual(w.clone().requires_grad_(), w))):
            with pytest.raises(RuntimeError, match="forward"):
                call()
        assert torch.equal(m(x, ids, w), m(x.clone(), ids, w)) and lin(v).shape == (9, 48)


def test_one_token_of_any_layout(route):
    """A single row, or logits of one dimension, whose experts are not neighbours in memory."""
    wide = _logits(6, 80)
    step("route of one token's strided logits")
    for x in (wide[2:3, ::2], wide[2, ::2], wide[:, 5:6].t(), wide[:, 5], wide.view(2, 3, 80)[1:, 1:2, ::4], wide[:1, ::2].double(), wide[2, :1]):
        top = min(3, x.shape[-1])
        ids, w = route(x, top)
        ref = route(x.contiguous(), top)
        assert ids.shape == (*x.shape[:-1], top) and torch.equal(ids, ref[0]) and torch.equal(w, ref[1])
        leaf = x.clone(memory_format=torch.contiguous_format).requires_grad_()
        base = wide.double() if x.dtype == torch.float64 else wide.clone()
        base.requires_grad_()
        view = base.as_strided(x.shape, x.stride(), x.storage_offset()) if x.dtype == F32 else base[:1, ::2]
        d = torch.randn_like(w)
        want, = torch.autograd.grad(route(leaf, top)[1], leaf, d)
        got, = torch.autograd.grad(route(view, top)[1], base, d)
        assert torch.equal(got[got != 0].sort()[0], want.reshape(-1)[want.reshape(-1) != 0].sort()[0])


def test_numbers_that_32_bits_do_not_hold(route):
    """Groups past 2^32 are refused, not taken for what is left of them; any true value renormalises."""
    from weight_only_bit_group_amd import binding as B
    l = _logits()
    step("route with numbers past 32 bits")
    for bad in (dict(groups=2 ** 32 + 1), dict(groups=2 ** 32 + 4, top_groups=2), dict(groups=4, top_groups=2 ** 32 + 2), dict(groups=-2 ** 32 + 1),
                dict(groups=0), dict(groups=65), dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(groups=4, top_groups=-2 ** 32 + 2)):
        for call in (lambda: route(l, 3, **bad), lambda: route(l.clone().requires_grad_(), 3, **bad), lambda: B.aq_moe_route(l, 3, **bad)):
            with pytest.raises(ValueError, match="groups"):
                call()
    ref = route(l, 3)
    for yes in (1, 2 ** 32, "yes"):
        assert torch.equal(route(l, 3, renormalize=yes)[1], ref[1])
    d = torch.randn(9, 3, device="cuda")
    assert torch.equal(B.aq_moe_route_backward(l, *ref, d, renormalize=2 ** 32), B.aq_moe_route_backward(l, *ref, d))
