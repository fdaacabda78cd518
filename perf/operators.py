"""Measured cases of the MXFP4 operators: quantising and reading back, products with 16-bit and with
MXFP4 activations, and the same products grouped by expert with ragged row counts.

MXFP4 is a block of 32 consecutive k of one row: E2M1 codes (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6; two
codes per byte, even k in the low nibble) and one E8M0 byte s, the factor 2^(s - 127).

``run`` makes the framework's calls where ``own`` is true and computes the plain form elsewhere;
``exact`` is the definition in 64 bits, written apart from both.
"""
import math

import torch

own = False

BLOCK = 32


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # the activations of a decode batch on their way into an MXFP4 product: the smallest call
        dict(name="quantize_decode_rows", op="quantize", m=16, k=2048, dtype="bf16"),
        # a whole fp32 weight matrix quantised when a checkpoint is loaded, and read back
        dict(name="quantize_weight_f32", op="quantize", m=14336, k=4096, dtype="f32"),
        # one token through a gate / up projection, activations kept in 16 bits
        dict(name="a16_one_token", op="gemm_a16", m=1, n=11008, k=2048, out="f32"),
        # a decode batch through a projection with long rows
        dict(name="a16_decode_batch", op="gemm_a16", m=16, n=4096, k=14336, out="f32"),
        # a prefill chunk, activations kept in 16 bits
        dict(name="a16_prefill", op="gemm_a16", m=4096, n=11008, k=2048, out="bf16"),
        # a short prompt: odd rows and columns, rows that end inside a tile of k
        dict(name="a4_short_prompt_odd", op="gemm_a4", m=333, n=1003, k=2080, out="bf16"),
        # a prefill chunk with the activations quantised too
        dict(name="a4_prefill", op="gemm_a4", m=4096, n=11008, k=2048, out="bf16"),
        # the same with longer rows and 32-bit outputs
        dict(name="a4_prefill_f32", op="gemm_a4", m=2048, n=14336, k=4096, out="f32"),
        # one token through its eight experts of 64
        dict(name="experts_a16_one_token", op="grouped_a16", t=1, top=8, e=64, n=1536, k=2048, gather=True,
             skew=0.5, out="bf16"),
        # a short prompt over experts of very different popularity, some without a row
        dict(name="experts_a16_ragged", op="grouped_a16", t=700, top=4, e=32, n=1408, k=2048, gather=True,
             skew=2.0, out="bf16"),
        # a decode batch over many experts, a few rows each; the second product (rows already grouped)
        dict(name="experts_a4_few_rows", op="grouped_a4", t=64, top=8, e=128, n=2048, k=1024, gather=False,
             skew=0.5, out="bf16"),
        # a prefill chunk over 64 experts
        dict(name="experts_a4_prefill", op="grouped_a4", t=4096, top=8, e=64, n=2048, k=2048, gather=True,
             skew=0.5, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm_a16", "gemm_a4", "grouped_a16", "grouped_a4"])
    k = BLOCK * _log(rng, 2, 448)
    if op == "quantize":
        m = min(_log(rng, 1, 16384), (14336 * 4096) // k)
        return dict(op=op, m=max(1, m), k=k, dtype=rng.choice(["bf16", "f32"]))
    out = rng.choice(["f32", "bf16"])
    n = _log(rng, 64, 14336)
    if op.startswith("gemm"):
        m = _log(rng, 1, 4096)
        while m * n * k > 4096 * 11008 * 2048:
            m = max(1, m // 2)
        return dict(op=op, m=m, n=n, k=k, out=out)
    e = _log(rng, 4, 128)
    top = rng.randint(1, min(8, e))
    while e * n * k > 64 * 2048 * 2048:
        n = max(64, n // 2) if n >= k or k <= 64 else n
        k = max(64, BLOCK * (k // 64)) if k > n else k
    t = _log(rng, 1, 4096)
    while t * top * n * k > 4096 * 8 * 2048 * 2048:
        t = max(1, t // 2)
    return dict(op=op, t=t, top=top, e=e, n=n, k=k, gather=rng.choice([True, False]), skew=rng.choice([0.0, 0.5, 2.0]),
                out=out)


_OUT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- inputs --------------------------------------------------------------------------------------

def _activations(g, m, k):
    """N(0, 1) rows with one channel in a hundred twenty times larger, bf16."""
    x = torch.randn(m, k, generator=g, device="cuda")
    big = torch.rand(k, generator=g, device="cuda") < 0.01
    return (x * (1.0 + 19.0 * big)).bfloat16()


def _weight(g, *shape):
    """Codes and scale bytes of N(0, 0.02) weights, as a checkpoint holds them."""
    w = torch.randn(*shape, generator=g, device="cuda") * 0.02
    mag, e = _round_blocks(w)
    neg = (w < 0) & (mag > 0)
    code = torch.bucketize(mag, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")).to(torch.uint8)
    code = code + 8 * neg.to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(op=op)
    if op == "quantize":
        x = _activations(g, case["m"], case["k"])
        s["x"] = x if case["dtype"] == "bf16" else x.float() * torch.rand(case["m"], 1, generator=g, device="cuda")
        return s
    s["out"] = _OUT[case["out"]]
    if op.startswith("gemm"):
        s["x"] = _activations(g, case["m"], case["k"])
        s["codes"], s["scales"] = _weight(g, case["n"], case["k"])
        return s
    t, top, e = case["t"], case["top"], case["e"]
    score = torch.randn(t, e, generator=g, device="cuda") + case["skew"] * torch.randn(e, generator=g, device="cuda")
    chosen = score.topk(top, dim=1).indices.reshape(-1)
    expert, order = torch.sort(chosen, stable=True)
    counts = torch.bincount(expert, minlength=e)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())
    s["rows"] = (order // top).to(torch.int32) if case["gather"] else None
    s["x"] = _activations(g, t if case["gather"] else t * top, case["k"])
    s["codes"], s["scales"] = _weight(g, e, case["n"], case["k"])
    return s


# ---- the plain form ------------------------------------------------------------------------------

def _round_blocks(x):
    """(E2M1 magnitudes, block exponents) of x [..., K]: the exponent is floor(log2(max |x|)) - 2, at least
    -127, and the magnitudes are |x| 2^-exponent at the nearest code, ties to the even one, at most 6."""
    a = x.float().abs().unflatten(-1, (-1, BLOCK))
    e = (torch.frexp(a.amax(-1))[1] - 3).clamp(min=-127)
    e = torch.where(a.amax(-1) == 0, -127, e)
    y = (a * ((127 - e) << 23).int().view(torch.float32).unsqueeze(-1)).flatten(-2)
    mag = 0.5 * (y > 0.25) + 0.5 * (y >= 0.75) + 0.5 * (y > 1.25) + 0.5 * (y >= 1.75)
    return mag + 1.0 * (y > 2.5) + 1.0 * (y >= 3.5) + 2.0 * (y > 5.0), e


def _power(e):
    """2^e for whole e from -127 up, without rounding."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _rounded(x):
    """x rounded to MXFP4, as the 32-bit values that its codes stand for."""
    mag, e = _round_blocks(x)
    v = torch.where(x < 0, -mag, mag)
    return (v.unflatten(-1, (-1, BLOCK)) * _power(e).unsqueeze(-1)).flatten(-2)


def _values(codes, scales):
    """The 32-bit values of codes [..., K/2] and scale bytes [..., K/32]."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * _power(scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _rounded(s["x"]).bfloat16()
    x = _rounded(s["x"]) if op.endswith("a4") else s["x"].float()
    w = _values(s["codes"], s["scales"])
    if op.startswith("gemm"):
        return (x @ w.t()).to(s["out"])
    # experts padded to the row count of the largest one, multiplied as a batch
    off = s["offsets"].long()
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    at = (off[:-1, None] + torch.arange(s["most"], device=x.device)).clamp(max=x.shape[0] - 1)
    y = torch.bmm(x[at], w.transpose(1, 2).contiguous())
    row = torch.arange(x.shape[0], device=x.device)
    expert = torch.searchsorted(off[1:].contiguous(), row, right=True)
    return y[expert, row - off[expert]].to(s["out"])


# ---- the framework's calls -----------------------------------------------------------------------

def _own(s):
    from weight_only_bit_group_amd import binding as B
    op = s["op"]
    if op == "quantize":
        return B.aq_mxfp4_dequantize(*B.aq_mxfp4_quantize(s["x"]), out_dtype=torch.bfloat16)
    if op == "gemm_a16":
        return B.aq_mxfp4_gemm(s["x"], s["codes"], s["scales"], out_dtype=s["out"])
    if op == "gemm_a4":
        xc, xs = B.aq_mxfp4_quantize(s["x"])
        return B.aq_mxfp4_gemm_a4(xc, xs, s["codes"], s["scales"], out_dtype=s["out"])
    if op == "grouped_a16":
        return B.aq_mxfp4_grouped_gemm(s["x"], s["codes"], s["scales"], s["offsets"], rows=s["rows"],
                                       out_dtype=s["out"])
    xc, xs = B.aq_mxfp4_quantize(s["x"])
    return B.aq_mxfp4_grouped_gemm_a4(xc, xs, s["codes"], s["scales"], s["offsets"], rows=s["rows"],
                                      out_dtype=s["out"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    """Bytes: each input once, each output once (the experts' weights that have a row, at most all)."""
    op, k = case["op"], case["k"]
    if op == "quantize":
        return dict(bytes=case["m"] * k * ((2 if case["dtype"] == "bf16" else 4) + 2), flops=2 * case["m"] * k)
    n, size = case["n"], 2 if case["out"] == "bf16" else 4
    packed = n * (k // 2 + k // BLOCK)
    if op.startswith("gemm"):
        return dict(bytes=packed + case["m"] * (2 * k + size * n), flops=2 * case["m"] * n * k)
    rows = case["t"] * case["top"]
    return dict(bytes=packed * min(case["e"], rows) + (case["t"] if case["gather"] else rows) * 2 * k + rows * size * n,
                flops=2 * rows * n * k)


# ---- the definition in 64 bits -------------------------------------------------------------------

def _exact_round(x):
    x = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top))
    # log2 may round up to a whole number just below a power of two
    e = torch.where(torch.pow(2.0, e) > top, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= top, e + 1, e)
    step = torch.pow(2.0, torch.where(top > 0, (e - 2).clamp(min=-127), torch.full_like(e, -127.0)))
    y = (x / step).clamp(-6, 6)
    # the grid has steps of .5 below 2, 1 below 4 and 2 above; torch.round takes ties to the even multiple
    grid = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return (torch.round(y / grid) * grid * step).flatten(-2)


def _exact_weight(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    m = torch.remainder(c, 8)
    mag = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(c >= 8, -mag, mag)
    return (v.unflatten(-1, (-1, BLOCK)) * torch.pow(2.0, scales.double() - 127).unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        return _exact_round(s["x"])
    x = _exact_round(s["x"]) if op.endswith("a4") else s["x"].double()
    if op.startswith("gemm"):
        return x @ _exact_weight(s["codes"], s["scales"]).t()
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    off = s["offsets"].tolist()
    y = torch.empty(x.shape[0], case["n"], dtype=torch.float64, device=x.device)
    for i in range(case["e"]):
        if off[i + 1] > off[i]:
            y[off[i]:off[i + 1]] = x[off[i]:off[i + 1]] @ _exact_weight(s["codes"][i], s["scales"][i]).t()
    return y
