"""route's gradient as a part of torch's graph: the native node and the Python function give the same, and both keep its rules."""
import gc

import pytest
import torch

from tests.gpu_util import step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class _Refuses:
    """Stands for the native module: calls go through Python; it still tells what a capture meets."""

    def __getattr__(self, name):
        if name == "capture_conflict":
            from weight_only_bit_group_amd import _aq_torch
            return _aq_torch.capture_conflict
        return lambda *a: None


@pytest.fixture(params=["native", "python"])
def route(request, monkeypatch):
    from weight_only_bit_group_amd import binding as B, layer
    if request.param == "python":
        monkeypatch.setattr(B, "_mx", _Refuses())
    step(f"route's graph, {request.param}")
    return layer.route


def _logits(t=9, e=24, dtype=torch.float32, seed=0):
    return torch.randn(t, e, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


HOWS = [dict(), dict(score="sigmoid", renormalize=False, scale=2.5), dict(renormalize=False), dict(score="sigmoid", groups=4, top_groups=2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("how", HOWS)
def test_gradient_is_the_binding_call(route, dtype, how):
    from weight_only_bit_group_amd import binding as B
    l = _logits(dtype=dtype).requires_grad_()
    held = l.detach().float() if dtype == torch.float64 else l.detach()
    ids, w = route(l, 3, bias=torch.zeros(24, device="cuda"), **how)
    assert not ids.requires_grad and w.requires_grad and w.grad_fn is not None
    rid, rw = B.aq_moe_route(held, 3, bias=torch.zeros(24, device="cuda"), **how)
    assert torch.equal(ids, rid) and torch.equal(w, rw)
    d = torch.randn_like(w)
    kept = {k: how[k] for k in ("score", "renormalize", "scale") if k in how}
    ref = B.aq_moe_route_backward(held, rid, rw, d, **kept).to(dtype)
    got, = torch.autograd.grad(w, l, d, retain_graph=True)
    assert got.dtype == dtype and torch.equal(got, ref)
    got, = torch.autograd.grad(w, l, d.t().contiguous().t())   # (a gradient that is not dense)
    assert torch.equal(got, ref)
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad(w, l, d)


def test_leading_dimensions_views_and_accumulation(route):
    l = _logits(12, 16).requires_grad_()
    ids, w = route(l.view(3, 4, 16), 2)
    assert ids.shape == w.shape == (3, 4, 2)
    w.square().sum().backward()
    one = l.grad.clone()
    (2 * route(l, 2)[1].square()).sum().backward()
    assert torch.allclose(l.grad, 3 * one, rtol=1e-6, atol=0)
    wide = _logits(8, 40).requires_grad_()
    _, w = route(wide[:, 5:29], 2)
    w[:, 0].sum().backward()
    assert (wide.grad[:, :5] == 0).all() and (wide.grad[:, 29:] == 0).all() and (wide.grad[:, 5:29] != 0).any()


def test_gradient_against_differences(route):
    """(f(l + h) - f(l - h)) / 2h of a random sum of the weights: the third derivative of the weights is below 2 scale, so the
    difference is off by h^2 / 3 scale and by two roundings of each weight, 2^-24 scale, over 2h; bounds of a sum of 5."""
    l = (4 * _logits(1, 12)).requires_grad_()
    h = 2.0 ** -7
    for how in (dict(), dict(score="sigmoid"), dict(renormalize=False), dict(score="sigmoid", renormalize=False)):
        ids, w = route(l, 5, **how)
        d = torch.rand_like(w) - 0.5
        g, = torch.autograd.grad(w, l, d)
        for e in range(12):
            step_ = torch.zeros_like(l)
            step_[0, e] = h
            hi, lo = (route((l + s).detach(), 5, bias=-1e3 * torch.ones(12, device="cuda").index_fill(0, ids[0].long(), 0), **how) for s in (step_, -step_))
            # (the same experts chosen by the bias, wherever the step moves the logits; in the order of ids)
            value = [(d[0] * torch.stack([ws[0][i[0] == x].sum() for x in ids[0]])).sum().double() for i, ws in (hi, lo)]
            diff = (value[0] - value[1]) / (2 * h)
            assert abs(float(diff - g[0, e])) <= 5 * (h * h / 3 * 2 + 2 ** -24 / h) + 2 ** -22


def test_no_gradient_of_the_gradient(route):
    l = _logits().requires_grad_()
    d = torch.randn(9, 3, device="cuda", requires_grad=True)
    _, w = route(l, 3)
    g, = torch.autograd.grad(w, l, d, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate"):
        g.sum().backward()
    _, w = route(l, 3)
    g, = torch.autograd.grad(w, l, d.detach(), create_graph=True)   # (nothing there asks for a gradient)
    assert torch.isfinite(g).all()


def test_changed_logits_are_noticed(route):
    a = _logits().requires_grad_()
    l = a * 1.0
    _, w = route(l, 3)
    l.detach().add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        w.sum().backward()
    _, w = route(a * 1.0, 3)
    w.detach().zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        w.sum().backward()


def test_grad_modes(route):
    l = _logits().requires_grad_()
    with torch.no_grad():
        assert not route(l, 3)[1].requires_grad
    with torch.inference_mode():
        assert not route(l, 3)[1].requires_grad and torch.equal(route(_logits(), 3)[0], route(l, 3)[0])
    seen = []
    _, w = route(l, 3)
    w.register_hook(lambda g: seen.append(g.clone()) or 2 * g)
    w.sum().backward()
    twice = l.grad.clone()
    l.grad = None
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.cpu(), lambda t: t.cuda()):
        _, w = route(l, 3)
    w.sum().backward()
    assert torch.allclose(twice, 2 * l.grad, rtol=1e-6, atol=1e-9) and (seen[0] == 1).all()
    ids, w = route(l, 3)
    assert (ids.float().sum() + w.detach().sum()).requires_grad is False


def test_backward_captured_and_replayed(route):
    """Forward and gradient in one captured graph, replayed with the program's own work between."""
    l, d = _logits(300, 64).requires_grad_(), torch.randn(300, 4, device="cuda")

    def call():
        ids, w = route(l, 4, score="sigmoid", groups=8, top_groups=3)
        return ids, w.detach(), *torch.autograd.grad(w, l, d)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = call()
    for i in range(3):
        with torch.no_grad():
            l.normal_()
            l[:, i] = float("-inf")
        d.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call()))


def test_capture_beside_a_living_graph_is_refused(route):
    """Leaves whose earlier graph lives on another stream: refused when the call is made, before anything is recorded."""
    from weight_only_bit_group_amd import layer
    l = _logits(20, 32).requires_grad_()
    m = layer.FP8Experts.from_weights(torch.randn(4, 64, 32, device="cuda"), torch.randn(4, 32, 32, device="cuda"))
    x, ids, w = torch.randn(20, 32, device="cuda"), torch.randint(0, 4, (20, 2), device="cuda"), torch.rand(20, 2, device="cuda").requires_grad_()
    alive = [route(l, 2)[1], route(l * 2.0, 2)[1], m(x, ids, w)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: route(l, 2), lambda: route(l * 2.0, 2), lambda: m(x, ids, w), lambda: m(x, ids, w * 0.5)):
        g = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="earlier call"):
            with torch.cuda.graph(g, stream=side):
                x.add_(0.0)   # (a graph of something)
                call()
    alive[0].sum().backward()
    del alive, call
    l.grad = w.grad = None
    gc.collect()   # (the refused calls' exceptions hold their frames, and these the graphs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):   # (let go: captured)
        out = torch.autograd.grad(route(l, 2)[1].square().sum(), l)[0], torch.autograd.grad(m(x, ids, w).square().sum(), w)[0]
    ref = torch.autograd.grad(route(l, 2)[1].square().sum(), l)[0], torch.autograd.grad(m(x, ids, w).square().sum(), w)[0]
    for _ in range(3):
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_backward_of_threads_at_once(route):
    from concurrent.futures import ThreadPoolExecutor

    def one(seed):
        l = _logits(200, 32, seed=seed).requires_grad_()
        with torch.cuda.stream(torch.cuda.Stream()):
            l2 = l.detach().clone().requires_grad_()
            out = []
            for _ in range(5):
                _, w = route(l2, 3)
                out.append(torch.autograd.grad(w.square().sum(), l2)[0])
            torch.cuda.current_stream().synchronize()
        return out

    torch.cuda.synchronize()
    with ThreadPoolExecutor(4) as pool:
        results = list(pool.map(one, range(8)))
    for seed, out in enumerate(results):
        l = _logits(200, 32, seed=seed).requires_grad_()
        _, w = route(l, 3)
        ref, = torch.autograd.grad(w.square().sum(), l)
        assert all(torch.equal(o, ref) for o in out)
