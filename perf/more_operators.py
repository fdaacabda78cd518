"""Measured cases of the FP8 operators and of the routing to experts: quantising and reading back, products of
16-bit activations with FP8 weights, the products grouped by expert, routing with its gradient, and the experts
of a mixture as a whole.

FP8 here is E4M3 (4 exponent and 3 mantissa bits, largest value 448) with one fp32 scale S for each block: 128
consecutive k of a row (activations) or 128 rows by 128 k (weights); the last block of a row or column may be
shorter.  With a the largest |x| of the block,

    S = max(fl32(a / 448), 2^-126),   code = the E4M3 value nearest to fl32(x / S), ties to the even code,

and a code stands for code * S.

``run`` makes the framework's calls where ``own`` is true and computes the plain form elsewhere; ``exact`` is the
definition in 64 bits, written apart from both.
"""
import math

import torch

own = False

BLOCK = 128


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the activations of a decode batch on their way into a product: the smallest call
        dict(name="quantize_decode_rows", op="quantize", m=16, k=2048, dtype="bf16", rows=1),
        # a whole fp32 weight matrix quantised in 128 x 128 blocks when a checkpoint is loaded, and read back
        dict(name="quantize_weight_f32", op="quantize", m=14336, k=4096, dtype="f32", rows=128),
        # one token through a gate / up projection
        dict(name="linear_one_token", op="linear", m=1, n=11008, k=2048, out="f32"),
        # a decode batch through a projection with long rows
        dict(name="linear_decode_batch", op="linear", m=32, n=4096, k=14336, out="bf16"),
        # a short prompt: odd rows and columns, a last block of 16 k
        dict(name="linear_short_prompt_odd", op="linear", m=333, n=1003, k=2064, out="f32"),
        # a prefill chunk
        dict(name="linear_prefill", op="linear", m=4096, n=11008, k=2048, out="bf16"),
        # a decode batch over many experts, a few rows each (rows already grouped)
        dict(name="grouped_few_rows", op="grouped", t=64, top=8, e=128, n=2048, k=1024, gather=False, skew=0.5,
             out="bf16"),
        # a prefill chunk over 64 experts
        dict(name="grouped_prefill", op="grouped", t=4096, top=8, e=64, n=2048, k=2048, gather=True, skew=0.5,
             out="bf16"),
        # a decode batch's routing over groups of experts, with a bias for balance and some experts masked
        dict(name="route_decode_groups", op="route", t=16, e=256, top=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renormalize=True, masked=True, dtype="f32", train=False),
        # a training step's routing and its gradient
        dict(name="route_train", op="route", t=16384, e=128, top=8, score="softmax", bias=False, groups=1,
             top_groups=1, renormalize=True, masked=False, dtype="bf16", train=True),
        # a decode batch through a mixture's experts
        dict(name="experts_decode", op="experts", t=16, top=8, e=64, k=2048, inner=1408, skew=0.5),
        # a prefill chunk through the same experts
        dict(name="experts_prefill", op="experts", t=2048, top=8, e=64, k=2048, inner=1408, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "grouped", "route", "experts"])
    if op == "quantize":
        k = 16 * _log(rng, 4, 896)
        m = max(1, min(_log(rng, 1, 16384), (14336 * 4096) // k))
        return dict(op=op, m=m, k=k, dtype=rng.choice(["bf16", "f32"]), rows=rng.choice([1, 128]))
    if op == "linear":
        m, n, k = _log(rng, 1, 4096), _log(rng, 64, 14336), 16 * _log(rng, 4, 896)
        while m * n * k > 4096 * 11008 * 2048:
            m = max(1, m // 2)
        return dict(op=op, m=m, n=n, k=k, out=rng.choice(["f32", "bf16"]))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        e = groups * _log(rng, 4, 512 // groups)
        score = rng.choice(["softmax", "sigmoid"])
        top = rng.randint(1, min(8, e // groups))
        t = max(1, min(_log(rng, 1, 16384), 16384 * 128 // e))
        return dict(op=op, t=t, e=e, top=top, score=score, bias=rng.choice([True, False]), groups=groups,
                    top_groups=rng.randint(1, groups), renormalize=rng.choice([True, False]),
                    masked=rng.choice([True, False]), dtype=rng.choice(["f32", "bf16"]),
                    train=rng.choice([True, False]))
    e = _log(rng, 4, 128)
    top = rng.randint(1, min(8, e))
    skew = rng.choice([0.0, 0.5, 2.0])
    t = _log(rng, 1, 4096)
    if op == "grouped":
        n, k = _log(rng, 64, 4096), 16 * _log(rng, 4, 256)
        while e * n * k > 64 * 2048 * 2048:
            n, k = max(64, n // 2) if n >= k else n, max(64, k // 32 * 16) if k > n else k
        while t * top * n * k > 4096 * 8 * 2048 * 2048:
            t = max(1, t // 2)
        return dict(op=op, t=t, top=top, e=e, n=n, k=k, gather=rng.choice([True, False]), skew=skew,
                    out=rng.choice(["f32", "bf16"]))
    k, inner = 16 * _log(rng, 4, 256), 16 * _log(rng, 4, 160)
    while e * k * inner > 64 * 2048 * 1408:
        k, inner = max(64, k // 32 * 16) if k >= inner else k, max(64, inner // 32 * 16) if inner > k else inner
    while t * top * k * inner > 2048 * 8 * 2048 * 1408:
        t = max(1, t // 2)
    return dict(op=op, t=t, top=top, e=e, k=k, inner=inner, skew=skew)


_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- inputs --------------------------------------------------------------------------------------

def _activations(g, m, k):
    """N(0, 1) rows with one channel in a hundred twenty times larger, bf16."""
    x = torch.randn(m, k, generator=g, device="cuda")
    big = torch.rand(k, generator=g, device="cuda") < 0.01
    return (x * (1.0 + 19.0 * big)).bfloat16()


def _weight(g, *shape):
    """Codes and block scales of N(0, 0.02) weights, as a checkpoint holds them."""
    c, s = _round_blocks(torch.randn(*shape, generator=g, device="cuda") * 0.02, BLOCK)
    return c.to(torch.float8_e4m3fn), s


def _choices(g, case):
    """A router's choices [t, top]: distinct experts, some far more popular than others."""
    score = torch.randn(case["t"], case["e"], generator=g, device="cuda")
    score = score + case["skew"] * torch.randn(case["e"], generator=g, device="cuda")
    return score.topk(case["top"], dim=1).indices


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(op=op)
    if op == "quantize":
        x = _activations(g, case["m"], case["k"])
        s["x"] = x if case["dtype"] == "bf16" else x.float() * torch.rand(case["m"], 1, generator=g, device="cuda")
        s["rows"], s["out"] = case["rows"], _TYPE[case["dtype"]]
        return s
    if op == "linear":
        s["out"] = _TYPE[case["out"]]
        s["x"] = _activations(g, case["m"], case["k"])
        s["codes"], s["scales"] = _weight(g, case["n"], case["k"])
        return s
    if op == "route":
        t, e = case["t"], case["e"]
        l = 1.5 * torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        if case["masked"]:   # one expert in ten, and every expert of one token in fifty
            off = torch.rand(t, e, generator=g, device="cuda") < 0.1
            off |= torch.rand(t, 1, generator=g, device="cuda") < 0.02
            l = l.masked_fill(off, float("-inf"))
        s["logits"] = l.to(_TYPE[case["dtype"]])
        s["bias"] = 0.1 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        s["grad"] = torch.randn(t, case["top"], generator=g, device="cuda") if case["train"] else None
        s["how"] = dict(score=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                        renormalize=case["renormalize"], scale=2.5)
        s["top"] = case["top"]
        return s
    ids = _choices(g, case)
    top, e = case["top"], case["e"]
    expert, order = torch.sort(ids.reshape(-1), stable=True)
    counts = torch.bincount(expert, minlength=e)
    s["most"] = int(counts.max())
    if op == "grouped":
        s["out"] = _TYPE[case["out"]]
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["rows"] = (order // top).to(torch.int32) if case["gather"] else None
        s["x"] = _activations(g, case["t"] * (1 if case["gather"] else top), case["k"])
        s["codes"], s["scales"] = _weight(g, e, case["n"], case["k"])
        return s
    s["ids"] = ids.to(torch.int32)
    s["weights"] = torch.softmax(torch.randn(case["t"], top, generator=g, device="cuda"), 1)
    s["x"] = _activations(g, case["t"], case["k"])
    s["gate_up"] = _weight(g, e, 2 * case["inner"], case["k"])
    s["down"] = _weight(g, e, case["k"], case["inner"])
    if own:
        from weight_only_bit_group_amd import layer
        s["module"] = layer.FP8Experts(*s["gate_up"], *s["down"], out_dtype=torch.bfloat16)
    return s


# ---- the plain form ------------------------------------------------------------------------------

def _padded(x, rows):
    """x [.., M, K] in blocks [.., Mb, rows, Kb, 128], filled up with zeros."""
    m, k = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -m % rows))
    return x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, rows))


def _cut(v, m, k):
    return v.flatten(-4, -3).flatten(-2)[..., :m, :k]


def _round_blocks(x, rows):
    """(E4M3 values [.., M, K] in 32 bits, scales [.., Mb, Kb]) of x [.., M, K]."""
    m, k = x.shape[-2:]
    b = _padded(x.float(), rows)
    top = b.abs().amax((-3, -1))
    s = (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -126)   # (by a number: times its rounded reciprocal)
    q = b / s[..., None, :, None]
    # steps of an eighth of the value's power of two, at least 2^-9; round takes ties to the even multiple
    e = (torch.frexp(q)[1] - 1).clamp(min=-6)
    step = ((e - 3 + 127) << 23).int().view(torch.float32)
    return _cut((torch.round(q / step) * step).clamp(-448.0, 448.0), m, k), s


def _values(codes, scales):
    """The 32-bit values of E4M3 values [.., M, K] and scales [.., Mb, Kb] (rows of a block: M / Mb, rounded up)."""
    m, k = codes.shape[-2:]
    rows = 1 if scales.shape[-2] == m else BLOCK
    return _cut(_padded(codes.float(), rows) * scales[..., None, :, None], m, k)


def _rounded(x):
    return _values(*_round_blocks(x, 1))


def _by_expert(x, w, at):
    """Rows x, as a batch of every expert's rows (at: [E, most] row numbers), times the experts' weights."""
    return torch.bmm(x[at], w.transpose(1, 2).contiguous())


def _plain_route(s):
    # in 64 bits: two experts' scores may lie within a 32-bit rounding of each other
    l = s["logits"].double()
    how, top = s["how"], s["top"]
    off = l == -math.inf
    empty = off.all(1, keepdim=True)
    if how["score"] == "softmax":
        p = torch.exp(l - torch.where(empty, 0.0, l.amax(1, keepdim=True)))
        p = p / torch.where(empty, 1.0, p.sum(1, keepdim=True))
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = p if s["bias"] is None else p + s["bias"].double()
    key = key.masked_fill(off, -math.inf)
    if how["groups"] > 1:
        best = torch.sort(key.unflatten(1, (how["groups"], -1)), dim=2, descending=True)[0][..., :2]
        score = torch.where((best == -math.inf).all(2), -math.inf, best.clamp(min=-1e300).masked_fill(best == -math.inf, 0.0).sum(2))
        order = torch.sort(score, dim=1, descending=True, stable=True)[1]
        out = torch.ones_like(score, dtype=torch.bool).scatter(1, order[:, :how["top_groups"]], False)
        key = key.masked_fill(out.repeat_interleave(key.shape[1] // how["groups"], 1), -math.inf)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    key, ids = key[:, :top], ids[:, :top]
    none = key == -math.inf
    chosen = torch.where(none, 0.0, p.gather(1, ids))
    total = chosen.sum(1, keepdim=True)
    share = torch.where(total > 0, chosen / torch.where(total > 0, total, 1.0), 0.0) if how["renormalize"] else chosen
    result = [torch.where(none, -1, ids).to(torch.int32), (how["scale"] * share).float()]
    if s["grad"] is not None:
        d = how["scale"] * s["grad"].double()
        mean = (share * d).sum(1, keepdim=True)
        if how["score"] == "softmax" and how["renormalize"]:
            dl = torch.zeros_like(l).scatter_add(1, ids, share * (d - mean))
        elif how["score"] == "softmax":
            dl = torch.zeros_like(l).scatter_add(1, ids, chosen * d) - p * mean
        else:
            if how["renormalize"]:
                d = torch.where(total > 0, (d - mean) / torch.where(total > 0, total, 1.0), 0.0)
            # (1 - sigmoid(l) as sigmoid(-l), which does not cancel)
            dl = torch.zeros_like(l).scatter_add(1, ids, torch.where(none, 0.0, d * chosen / (1.0 + torch.exp(l.gather(1, ids)))))
        result.append(dl.to(s["logits"].dtype))
    return result


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _values(*_round_blocks(s["x"], s["rows"])).to(s["out"])
    if op == "linear":
        return (_rounded(s["x"]) @ _values(s["codes"], s["scales"]).t()).to(s["out"])
    if op == "route":
        return _plain_route(s)
    x = _rounded(s["x"])
    if op == "grouped":
        off, w = s["offsets"].long(), _values(s["codes"], s["scales"])
        x = x if s["rows"] is None else x[s["rows"].long()]
        row = torch.arange(x.shape[0], device=x.device)
        expert = torch.searchsorted(off[1:].contiguous(), row, right=True)
        at = (off[:-1, None] + torch.arange(s["most"], device=x.device)).clamp(max=x.shape[0] - 1)
        return _by_expert(x, w, at)[expert, row - off[expert]].to(s["out"])
    # the experts: choices sorted by expert, each expert's padded to the most popular one's, as a batch
    t, top = s["ids"].shape
    e = s["gate_up"][0].shape[0]
    expert, order = torch.sort(s["ids"].reshape(-1), stable=True)
    off = torch.searchsorted(expert, torch.arange(e, device=x.device, dtype=expert.dtype))
    slot = torch.arange(t * top, device=x.device) - off[expert.long()]
    at = (off[:, None] + torch.arange(s["most"], device=x.device)).clamp(max=t * top - 1)
    h = _by_expert(x[order // top], _values(*s["gate_up"]), at)
    gate, up = h.chunk(2, dim=2)
    h = _rounded(gate / (1.0 + torch.exp(-gate)) * up)
    y = torch.bmm(h, _values(*s["down"]).transpose(1, 2).contiguous())
    back = torch.empty_like(order).scatter(0, order, torch.arange(t * top, device=x.device))
    y = y[expert.long()[back], slot[back]].view(t, top, -1)
    return (y * s["weights"][:, :, None]).sum(1).bfloat16()


# ---- the framework's calls -----------------------------------------------------------------------

def _own(s):
    from weight_only_bit_group_amd import binding as B, layer
    op = s["op"]
    if op == "quantize":
        codes, scales = B.aq_fp8_quantize(s["x"], block_rows=s["rows"])
        return B.aq_fp8_dequantize(codes, scales, block_rows=s["rows"], out_dtype=s["out"])
    if op == "linear":
        return B.aq_fp8_linear(s["x"], s["codes"], s["scales"], out_dtype=s["out"])
    if op == "grouped":
        codes, scales = B.aq_fp8_quantize(s["x"])
        return B.aq_fp8_grouped_gemm(codes, scales, s["codes"], s["scales"], s["offsets"], rows=s["rows"],
                                     out_dtype=s["out"])
    if op == "route":
        if s["grad"] is None:
            return list(layer.route(s["logits"], s["top"], bias=s["bias"], **s["how"]))
        logits = s["logits"].detach().requires_grad_()
        ids, weights = layer.route(logits, s["top"], bias=s["bias"], **s["how"])
        return [ids, weights.detach(), *torch.autograd.grad(weights, logits, s["grad"])]
    return s["module"](s["x"], s["ids"], s["weights"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def _packed(n, k):
    return n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK)


def work(case):
    """Bytes: each input once, each output once (the experts' weights that have a row, at most all)."""
    op = case["op"]
    if op == "quantize":
        return dict(bytes=2 * case["m"] * case["k"] * (2 if case["dtype"] == "bf16" else 4), flops=4 * case["m"] * case["k"])
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(bytes=_packed(n, k) + 2 * m * k + (2 if case["out"] == "bf16" else 4) * m * n, flops=2 * m * n * k)
    if op == "route":
        size = (2 if case["dtype"] == "bf16" else 4) * case["t"] * case["e"]
        small = case["t"] * case["top"]
        return dict(bytes=size * (2 if case["train"] else 1) + small * (12 if case["train"] else 8),
                    flops=case["t"] * case["e"] * (8 if case["train"] else 4))
    rows, k = case["t"] * case["top"], case["k"]
    seen = min(case["e"], rows)
    if op == "grouped":
        return dict(bytes=_packed(case["n"], k) * seen + (case["t"] if case["gather"] else rows) * 2 * k
                    + rows * case["n"] * (2 if case["out"] == "bf16" else 4), flops=2 * rows * case["n"] * k)
    inner = case["inner"]
    return dict(bytes=(_packed(2 * inner, k) + _packed(k, inner)) * seen + 4 * case["t"] * k + 8 * rows,
                flops=6 * rows * k * inner)


# ---- the definition in 64 bits -------------------------------------------------------------------

def _exact_values(x, rows):
    """x [M, K] rounded to FP8, block after block of k.  The scale and the quotient are fp32 by definition."""
    x = x.double()
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK):
        b = x[:, lo:lo + BLOCK]
        top = b.abs().amax(1)
        if rows > 1:
            top = torch.cat([part.amax().expand(part.shape[0]) for part in top.split(rows)])
        s = (top / torch.full_like(top, 448)).float().double().clamp(min=2.0 ** -126)[:, None]
        q = (b / s).float().double()
        mag = q.abs()
        grid = torch.full_like(mag, 2.0 ** -9)
        for power in range(-5, 9):   # from 2^power on the steps are 2^(power - 3)
            grid = torch.where(mag >= 2.0 ** power, 2.0 ** (power - 3), grid)
        out[:, lo:lo + BLOCK] = (torch.round(q / grid) * grid).clamp(-448, 448) * s
    return out


def _exact_weight(codes, scales):
    n, k = codes.shape
    s = scales.double().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return codes.float().double() * s


def _exact_route(case, s):
    l = s["logits"].double()
    t, e = l.shape
    off = torch.isneginf(l)
    if case["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    else:
        p = torch.sigmoid(l)
    key = torch.where(off, -math.inf, p if s["bias"] is None else p + s["bias"].double())
    if case["groups"] > 1:
        size = e // case["groups"]
        score = torch.full((t, case["groups"]), -math.inf, dtype=torch.float64, device=l.device)
        for j in range(case["groups"]):
            part = key[:, j * size:(j + 1) * size]
            first, at = part.max(1)
            second = part.scatter(1, at[:, None], -math.inf).max(1)[0]
            score[:, j] = torch.where(torch.isneginf(second), first, first + second)
        rank = torch.zeros_like(score)   # groups ahead of this one
        for j in range(case["groups"]):
            rank += score[:, j:j + 1] > score
            rank[:, j + 1:] += (score[:, j:j + 1] == score[:, j + 1:])
        key = torch.where((rank >= case["top_groups"]).repeat_interleave(size, 1), -math.inf, key)
    w = torch.zeros(t, case["top"], dtype=torch.float64, device=l.device)
    mask = torch.zeros(t, e, dtype=torch.float64, device=l.device)
    at = torch.zeros(t, case["top"], dtype=torch.long, device=l.device)
    for j in range(case["top"]):
        best = key.amax(1, keepdim=True)
        i = (key == best).double().argmax(1, keepdim=True)
        found = ~torch.isneginf(best)
        w[:, j:j + 1] = torch.where(found, p.gather(1, i), 0.0)
        mask.scatter_add_(1, i, found.double())
        at[:, j:j + 1] = torch.where(found, i, -1)
        key = key.scatter(1, i, -math.inf)
    total = w.sum(1, keepdim=True)
    if case["renormalize"]:
        weights = 2.5 * torch.nan_to_num(w / total, nan=0.0)
    else:
        weights = 2.5 * w
    result = [at.to(torch.int32), weights]
    if case["train"]:
        # the weights as a function of the logits at fixed choices, by the chain rule's Jacobian-vector product
        g = torch.zeros(t, e, dtype=torch.float64, device=l.device)
        for j in range(case["top"]):
            g.scatter_add_(1, at[:, j:j + 1].clamp(min=0), torch.where(at[:, j:j + 1] >= 0, s["grad"][:, j:j + 1].double(), 0.0))
        dp = 2.5 * g * mask
        if case["renormalize"]:
            dp = torch.nan_to_num((dp - mask * (dp * p).sum(1, keepdim=True) / total) / total, nan=0.0, posinf=0.0, neginf=0.0)
        dl = p * (dp - (p * dp).sum(1, keepdim=True)) if case["score"] == "softmax" else dp * p * torch.sigmoid(-l)
        result.append(torch.where(off, 0.0, dl))
    return result


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(s["x"], case["rows"])
    if op == "linear":
        return _exact_values(s["x"], 1) @ _exact_weight(s["codes"], s["scales"]).t()
    if op == "route":
        return _exact_route(case, s)
    x = _exact_values(s["x"], 1)
    if op == "grouped":
        x = x if s["rows"] is None else x[s["rows"].long()]
        off = s["offsets"].tolist()
        y = torch.empty(x.shape[0], case["n"], dtype=torch.float64, device=x.device)
        for i in range(case["e"]):
            if off[i + 1] > off[i]:
                y[off[i]:off[i + 1]] = x[off[i]:off[i + 1]] @ _exact_weight(s["codes"][i], s["scales"][i]).t()
        return y
    y = torch.zeros_like(x)
    for i in range(case["e"]):
        t, j = torch.nonzero(s["ids"] == i, as_tuple=True)
        if len(t):
            h = x[t] @ _exact_weight(s["gate_up"][0][i], s["gate_up"][1][i]).t()
            h = torch.sigmoid(h[:, :case["inner"]]) * h[:, :case["inner"]] * h[:, case["inner"]:]
            # (its block maxima and quotients are rounded as those of an fp32 input)
            o = _exact_values(h.float(), 1) @ _exact_weight(s["down"][0][i], s["down"][1][i]).t()
            y[t] += s["weights"].double()[t, j][:, None] * o
    return y
