"""Quantized linear module and the norm-group AWQ apply step, on top of the binding.

Every computation is a libaq call (pack, abs-mean, alpha search, GEMV / GEMM);
this module only arranges tensors and swaps modules.

  * ``W4A16Linear``: the drop-in replacement of an ``nn.Linear`` holding the
    packed INT4 triple; its forward is the W4A16 GEMV (M <= 16 rows) or GEMM
    ("Lance-Quant", zingnex.cn, "运行时替换与内存优化": linears replaced by
    quantized linear modules; "模型量化指南", blog.yoooo.fun, "共同约定": the
    quantized layer dequantizes in memory and equals the original layer with W
    replaced by its dequantized value, and quantizing an already quantized
    layer is refused).
  * ``norm_group_awq``: AWQ for one normalisation and the linears consuming its
    output ("Lance-Quant", "量化应用：网格搜索与分组策略": grid search of the
    scale per norm and its consumers, the scale folded into the preceding
    RMSNorm, group-wise INT4 packing).  The consumers are searched jointly:
    their weights concatenated along N share one channel scale s, the norm
    weight becomes w / s and each linear holds Q(W diag(s)).
  * ``quantize_linear``: plain group-wise min-max packing for linears with no
    norm in front of them (o_proj and down_proj follow a non-linearity, so no
    scale can be folded; same page, after the fourth case).
  * ``W8A16Linear`` and ``quantize_modules`` with ``LayerQuantPolicy``: the mixed
    4/8-bit policy ("模型量化指南", "混合精度（按层 4/8-bit）": a policy binds bits /
    group size / symmetry to named layers, unspecified fields inherit the base
    configuration, and a policy target outside the layers selected by
    target_modules is an error at parse time; "共同约定": explicit errors for a
    model without linears, targets that match nothing, and re-quantization).
  * ``MXFP4Linear`` and ``MXFP4Experts``: weights in MXFP4 blocks of 32, the
    activations kept in bf16 or quantized to MXFP4 on the way in; the experts of
    a mixture run as two products grouped by expert.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B


class W4A16Linear(torch.nn.Module):
    """y = x W^T (+ bias) with W stored as group-wise INT4 (packed [N, K/2], S, z).

    The input is cast to bf16 (the kernels' activation type); the output is fp32.
    """

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group: int,
                 bias: torch.Tensor | None = None):
        super().__init__()
        if packed.dim() != 2 or scales.shape != zeros.shape or scales.shape[0] != packed.shape[0]:
            raise ValueError("packed [N, K/2], scales and zeros [N, K/group] expected")
        self.group = int(group)
        self.in_features = packed.shape[1] * 2
        self.out_features = packed.shape[0]
        if scales.shape[1] * self.group != self.in_features:
            raise ValueError("scales must be [N, K/group]")
        self.register_buffer("packed", packed.contiguous())
        self.register_buffer("scales", scales.contiguous())
        self.register_buffer("zeros", zeros.contiguous())
        self.register_buffer("bias", None if bias is None else bias.detach().float().contiguous())
        self.split_sizes = [self.out_features]

    @classmethod
    def from_weight(cls, weight: torch.Tensor, group: int, chan_scale: torch.Tensor | None = None,
                    bias: torch.Tensor | None = None, sym: bool = False) -> "W4A16Linear":
        """Pack W [N, K] (fp32 or bf16, on the GPU), optionally scaled by chan_scale [K];
        sym=True packs the symmetric variant (same format, zero point 8)."""
        p, s, z = B.aq_quantize_pack(weight.detach().contiguous(), group, chan_scale, sym=sym)
        return cls(p, s, z, group, bias)

    @classmethod
    def concat(cls, mods) -> "W4A16Linear":
        """One module over the stacked output rows of several W4A16Linear with the same input
        size and group (the consumers of one norm, e.g. q|k|v or gate|up): one GEMV / GEMM
        launch instead of one per module.  Output rows are computed independently, so each
        slice of the result equals the separate module's output; ``split_sizes`` gives the
        slice widths (``torch.split(y, m.split_sizes, -1)``)."""
        mods = list(mods)
        if not mods:
            raise ValueError("nothing to concatenate")
        k, g = mods[0].in_features, mods[0].group
        for m in mods:
            if not isinstance(m, W4A16Linear):
                raise TypeError(f"expected W4A16Linear, got {type(m).__name__}")
            if m.in_features != k or m.group != g:
                raise ValueError("modules must share in_features and group")
        bias = None
        if any(m.bias is not None for m in mods):
            bias = torch.cat([m.bias if m.bias is not None else
                              torch.zeros(m.out_features, dtype=torch.float32, device=m.packed.device) for m in mods])
        out = cls(torch.cat([m.packed for m in mods]), torch.cat([m.scales for m in mods]),
                  torch.cat([m.zeros for m in mods]), g, bias)
        out.split_sizes = [m.out_features for m in mods]
        return out

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected {self.in_features} input features, got {x.shape[-1]}")
        x2 = x.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        m = x2.shape[0]
        if m <= 16:
            y = B.aq_w4a16_gemv(x2, self.packed, self.scales, self.zeros, self.group)
        else:
            # the staging matrix (as large as a bf16 copy of W) is allocated per call: torch's
            # caching allocator hands the block back in stream order, and no module keeps one
            y = B.aq_w4a16_gemm(x2, self.packed, self.scales, self.zeros, self.group)
        if self.bias is not None:
            y = y + self.bias
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, group={self.group}"


def _weight_of(linear) -> torch.Tensor:
    if isinstance(linear, (W4A16Linear, MXFP4Linear)):
        raise ValueError("layer is already quantized")
    if not isinstance(linear, torch.nn.Linear):
        raise TypeError(f"expected torch.nn.Linear, got {type(linear).__name__}")
    return linear.weight.detach()


def quantize_linear(linear: torch.nn.Linear, group: int, sym: bool = False) -> W4A16Linear:
    """Plain group-wise INT4 of one linear (no channel scale): min-max asymmetric, or
    symmetric (max |w| / 7, zero point 8) with sym=True."""
    w = _weight_of(linear)
    return W4A16Linear.from_weight(w.contiguous(), group, None, linear.bias, sym)


def norm_group_awq(norm_weight: torch.Tensor, linears, x_norm: torch.Tensor, group: int, n_grid: int = 20,
                   search_tokens: int = 4096):
    """AWQ of the linears consuming one RMSNorm's output.

    x_norm: that norm's output over the calibration tokens [T, K] bf16 (all T
    tokens give the abs-mean statistic; the first ``search_tokens`` score the
    search).  Returns (folded fp32 norm weight [K], [W4A16Linear per linear],
    search dict of aq_awq_search).
    """
    ws = [_weight_of(l) for l in linears]
    if not ws:
        raise ValueError("no linear to quantize")
    k = ws[0].shape[1]
    if any(w.shape[1] != k for w in ws) or any(w.dtype != ws[0].dtype for w in ws):
        raise ValueError("the consumers of one norm must share K and the weight dtype")
    if x_norm.dim() != 2 or x_norm.shape[1] != k:
        raise ValueError(f"x_norm must be [T, {k}]")
    t = x_norm.shape[0]
    x = x_norm.to(torch.bfloat16).contiguous()
    sum_abs = torch.zeros(k, dtype=torch.float64, device=x.device)
    mean = torch.empty(k, dtype=torch.float32, device=x.device)
    B.aq_act_absmean(x, sum_abs, t, mean)          # EINVAL (ValueError) for T == 0
    w_cat = torch.cat(ws, dim=0).contiguous()
    res = B.aq_awq_search(x[:search_tokens].contiguous(), mean.cpu(), w_cat, group, n_grid)
    folded = B.aq_awq_fold_norm(norm_weight.detach().contiguous(), res["best_scale"])
    out, n0 = [], 0
    for lin, w in zip(linears, ws):
        n1 = n0 + w.shape[0]
        out.append(W4A16Linear(res["packed"][n0:n1], res["scales"][n0:n1], res["zeros"][n0:n1], group, lin.bias))
        n0 = n1
    return folded, out, res


class W8A16Linear(torch.nn.Module):
    """y = x W^T (+ bias) with W stored as group-wise INT8 (codes [N, K], S, z); bf16 in, fp32 out."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group: int,
                 bias: torch.Tensor | None = None):
        super().__init__()
        if codes.dim() != 2 or scales.shape != zeros.shape or scales.shape[0] != codes.shape[0]:
            raise ValueError("codes [N, K], scales and zeros [N, K/group] expected")
        self.group = int(group)
        self.in_features = codes.shape[1]
        self.out_features = codes.shape[0]
        if scales.shape[1] * self.group != self.in_features:
            raise ValueError("scales must be [N, K/group]")
        self.register_buffer("codes", codes.contiguous())
        self.register_buffer("scales", scales.contiguous())
        self.register_buffer("zeros", zeros.contiguous())
        self.register_buffer("bias", None if bias is None else bias.detach().float().contiguous())

    @classmethod
    def from_weight(cls, weight: torch.Tensor, group: int, chan_scale: torch.Tensor | None = None,
                    bias: torch.Tensor | None = None) -> "W8A16Linear":
        c, s, z = B.aq_quantize_pack8(weight.detach().contiguous(), group, chan_scale)
        return cls(c, s, z, group, bias)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected {self.in_features} input features, got {x.shape[-1]}")
        x2 = x.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        m = x2.shape[0]
        if m <= 16:
            y = B.aq_w8a16_gemv(x2, self.codes, self.scales, self.zeros, self.group)
        else:
            # per-call staging matrix, as for W4A16Linear
            y = B.aq_w8a16_gemm(x2, self.codes, self.scales, self.zeros, self.group)
        if self.bias is not None:
            y = y + self.bias
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, group={self.group}, bits=8"


def _mx_act(act: str) -> str:
    if act not in ("bf16", "mxfp4"):
        raise ValueError(f"act must be 'bf16' or 'mxfp4' (got {act!r})")
    return act


def _mx_pair(codes: torch.Tensor, scales: torch.Tensor, name: str, ndim: int) -> None:
    """Checks codes [.., N, K/2] and scales [.., N, K/32], both uint8."""
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError(f"{name}: codes and scales must be uint8")
    if codes.dim() != ndim or codes.shape[-1] == 0 or codes.shape[-1] % 16 \
            or scales.shape != (*codes.shape[:-1], codes.shape[-1] // 16):
        raise ValueError(f"{name}: codes [.., N, K/2] and scales [.., N, K/32] expected "
                         f"(got {list(codes.shape)} and {list(scales.shape)})")


def _mx_rounded(x2: torch.Tensor, act: str):
    """The product's activation arguments: bf16 rows, or the codes and scales of rows in their own type."""
    if act == "bf16":
        return (x2.to(torch.bfloat16),)
    return B.aq_mxfp4_quantize(x2 if x2.dtype in (torch.bfloat16, torch.float32) else x2.float())


def _mx_rows(x: torch.Tensor, k: int) -> torch.Tensor:
    """x [.., K] as a matrix whose rows start at 16-byte addresses, copied only if they do not."""
    if x.shape[-1] != k:
        raise ValueError(f"expected {k} input features, got {x.shape[-1]}")
    x2 = x.reshape(-1, k)
    size = x2.element_size()
    if x2.stride(1) != 1 or x2.stride(0) < k or x2.stride(0) * size % 16 or x2.data_ptr() % 16:
        x2 = x2.contiguous()
        if x2.data_ptr() % 16:   # a dense slice that starts off the alignment
            x2 = x2.clone()
    return x2


class _NoBackward(torch.autograd.Function):
    """compute(x), whose gradient is refused when it is asked for."""

    @staticmethod
    def forward(ctx, name, compute, x):
        ctx.name = name
        return compute(x)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError(f"{ctx.name} has no backward pass: the gradient of its input is not computed "
                           "(run it under torch.no_grad(), or detach its input)")


def _forward_only(name: str, compute, x: torch.Tensor) -> torch.Tensor:
    """compute(x), a fresh tensor; part of the graph where x is, so that no gradient is lost in silence."""
    if torch.is_grad_enabled() and x.requires_grad:
        return _NoBackward.apply(name, compute, x)
    return compute(x)


class MXFP4Linear(torch.nn.Module):
    """y = x W^T (+ bias) with W in MXFP4 (codes [N, K/2], scales [N, K/32]).

    act="bf16" casts the input to bf16; act="mxfp4" quantizes it row by row to MXFP4, which
    runs on the block-scaled matrix instructions (four times the bf16 rate, coarser inputs).
    The output is fp32.  There is no backward pass: an input that requires a gradient gets its
    output, and an error when the gradient is asked for.
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
                 act: str = "bf16"):
        super().__init__()
        _mx_pair(codes, scales, "MXFP4Linear", 2)
        self.act = _mx_act(act)
        self.in_features = codes.shape[1] * 2
        self.out_features = codes.shape[0]
        self.register_buffer("codes", codes.contiguous())
        self.register_buffer("scales", scales.contiguous())
        self.register_buffer("bias", None if bias is None else bias.detach().float().contiguous())

    @classmethod
    def from_weight(cls, weight: torch.Tensor, bias: torch.Tensor | None = None, act: str = "bf16") -> "MXFP4Linear":
        """Quantize W [N, K] (fp32 or bf16, on the GPU; K a multiple of 32)."""
        _mx_act(act)
        return cls(*B.aq_mxfp4_quantize(weight.detach().contiguous()), bias, act)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        product = B.aq_mxfp4_gemm if self.act == "bf16" else B.aq_mxfp4_gemm_a4
        y = _forward_only("MXFP4Linear", lambda x2: product(*_mx_rounded(x2, self.act), self.codes, self.scales),
                          _mx_rows(x, self.in_features))
        if self.bias is not None:
            y += self.bias
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, weights=mxfp4, act={self.act}"


# torch's sort clears counters with memory-fill nodes above this size, which a graph's later replays
# do not repeat faithfully; below it a captured call has kernels and copies on the device only.
_CAPTURED_CHOICES = 1 << 20


class MXFP4Experts(torch.nn.Module):
    """The experts of a mixture, gated MLPs with MXFP4 weights:

        y[t] = sum_j w[t, j] D_e (silu(G_e x[t]) * (U_e x[t])),   e = ids[t, j]

    gate_up holds [G_e; U_e] as codes [E, 2I, K/2] and scales [E, 2I, K/32], down D_e as codes
    [E, K, I/2] and scales [E, K, I/32].  ``forward(x, ids, weights)`` takes x [.., K] with the
    router's choices ids [.., top] (any integer type) and weights [.., top]; a choice outside
    0 .. E - 1 (the filling of a padded batch, an expert of another rank) adds nothing.
    Both layers run as one product grouped by expert each, for all tokens, without reading a
    count back to the host.  A token's products are added in the order of its choices, in
    fp32: the result does not depend on how its choices were grouped.  The output is fp32.
    weights are differentiable, the experts are not: an error when x's gradient is asked for.
    A call may be captured into a graph up to 2^20 choices, and its replays follow x, ids and weights.
    """

    def __init__(self, gate_up_codes: torch.Tensor, gate_up_scales: torch.Tensor, down_codes: torch.Tensor,
                 down_scales: torch.Tensor, act: str = "bf16"):
        super().__init__()
        _mx_pair(gate_up_codes, gate_up_scales, "gate_up", 3)
        _mx_pair(down_codes, down_scales, "down", 3)
        self.act = _mx_act(act)
        self.num_experts, rows, half = gate_up_codes.shape
        self.features, self.inner = 2 * half, 2 * down_codes.shape[2]
        if rows != 2 * self.inner or tuple(down_codes.shape[:2]) != (self.num_experts, self.features):
            raise ValueError(f"gate_up [E, 2I, K] and down [E, K, I] expected, codes are {list(gate_up_codes.shape)} "
                             f"and {list(down_codes.shape)}")
        self.register_buffer("gate_up_codes", gate_up_codes.contiguous())
        self.register_buffer("gate_up_scales", gate_up_scales.contiguous())
        self.register_buffer("down_codes", down_codes.contiguous())
        self.register_buffer("down_scales", down_scales.contiguous())

    @classmethod
    def from_weights(cls, gate_up: torch.Tensor, down: torch.Tensor, act: str = "bf16") -> "MXFP4Experts":
        """Quantize gate_up [E, 2I, K] and down [E, K, I] (fp32 or bf16, on the GPU)."""
        _mx_act(act)
        pairs = []
        for w, name in ((gate_up, "gate_up"), (down, "down")):
            if w.dim() != 3:
                raise ValueError(f"{name} must have 3 dimensions")
            codes, scales = B.aq_mxfp4_quantize(w.detach().reshape(-1, w.shape[2]).contiguous())
            pairs += [codes.view(*w.shape[:2], -1), scales.view(*w.shape[:2], -1)]
        return cls(*pairs, act)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        x2 = _mx_rows(x, self.features)
        t = x2.shape[0]
        if ids.shape != weights.shape or ids.shape[:-1] != x.shape[:-1] or ids.dim() < 1 or ids.shape[-1] == 0:
            raise ValueError(f"ids and weights must be {[*x.shape[:-1], 'top']} (got {list(ids.shape)} and "
                             f"{list(weights.shape)})")
        if ids.is_floating_point() or ids.dtype == torch.bool:
            raise ValueError(f"ids must be integers (got {ids.dtype})")
        top = ids.shape[-1]
        flat = ids.reshape(-1).long()
        if flat.shape[0] > _CAPTURED_CHOICES and torch.cuda.is_current_stream_capturing():
            raise RuntimeError(f"MXFP4Experts: at most {_CAPTURED_CHOICES} choices in a captured call (got {flat.shape[0]})")
        valid = (flat >= 0) & (flat < self.num_experts)
        # choices sorted by expert, those outside the range behind the last one
        key, order = torch.where(valid, flat, self.num_experts).sort(stable=True)
        edges = torch.arange(self.num_experts + 1, device=key.device, dtype=key.dtype)
        offsets = torch.searchsorted(key, edges, out_int32=True)
        rows = (order // top).int()
        product = B.aq_mxfp4_grouped_gemm if self.act == "bf16" else B.aq_mxfp4_grouped_gemm_a4

        def experts(x2):
            h = product(*_mx_rounded(x2, self.act), self.gate_up_codes, self.gate_up_scales, offsets, rows)
            h = torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]
            return product(*_mx_rounded(h, self.act), self.down_codes, self.down_scales, offsets)

        y = _forward_only("MXFP4Experts", experts, x2)
        back = torch.empty_like(order)
        back[order] = torch.arange(order.shape[0], device=order.device)
        # (the rows behind the last expert were never written, and nothing is said of their weights)
        y = torch.where(valid[:, None], y[back], 0.0).view(t, top, self.features)
        w = torch.where(valid, weights.reshape(-1).float(), 0.0).view(t, top, 1)
        out = y[:, 0] * w[:, 0]
        for j in range(1, top):
            out += y[:, j] * w[:, j]
        return out.reshape(*x.shape[:-1], self.features)

    def extra_repr(self) -> str:
        return f"experts={self.num_experts}, features={self.features}, inner={self.inner}, weights=mxfp4, act={self.act}"


@dataclass(frozen=True)
class LayerQuantPolicy:
    """Per-layer override of the base configuration; None fields inherit it."""
    target_modules: tuple
    bits: int | None = None
    group_size: int | None = None
    sym: bool | None = None


def _matches(name: str, target: str) -> bool:
    """target names whole dotted components of name (a linear or one of its parents)."""
    return ("." + target + ".") in ("." + name + ".")


def plan_quantization(model: torch.nn.Module, target_modules, bits: int = 4, group_size: int = 64,
                      sym: bool = False, layer_policies=()):
    """{linear name: (bits, group_size, sym)} for the linears the call would quantize.

    Checks everything before anything is quantized: the model has linears, the
    targets match some, no target is already quantized, every policy target matches
    a selected linear, and every (bits, sym) pair is supported (4-bit asymmetric or
    symmetric, 8-bit asymmetric).
    """
    named = dict(model.named_modules())
    quantized = [n for n, m in named.items() if isinstance(m, (W4A16Linear, W8A16Linear, MXFP4Linear))]
    linears = [n for n, m in named.items() if isinstance(m, torch.nn.Linear)]
    if not linears and not quantized:
        raise ValueError("the model contains no torch.nn.Linear")
    targets = tuple(target_modules)
    hit = [n for n in linears if any(_matches(n, t) for t in targets)]
    again = [n for n in quantized if any(_matches(n, t) for t in targets)]
    if again:
        raise ValueError(f"already quantized: {again[0]}")
    if not hit:
        raise ValueError(f"target_modules {targets} match no linear")
    plan = {n: (bits, group_size, sym) for n in hit}
    for pol in layer_policies:
        sel = [n for n in hit if any(_matches(n, t) for t in pol.target_modules)]
        if not sel:
            raise ValueError(f"policy targets {tuple(pol.target_modules)} match no selected linear")
        for n in sel:
            b, g, s = plan[n]
            plan[n] = (pol.bits if pol.bits is not None else b, pol.group_size if pol.group_size is not None else g,
                       pol.sym if pol.sym is not None else s)
    for n, (b, g, s) in plan.items():
        if b not in (4, 8) or (b == 8 and s) or g not in (32, 64, 128):
            raise ValueError(f"{n}: unsupported configuration bits={b} group_size={g} sym={s}")
        k = named[n].in_features
        if k % g:
            raise ValueError(f"{n}: in_features {k} is not a multiple of group_size {g}")
    return plan


def quantize_modules(model: torch.nn.Module, target_modules, bits: int = 4, group_size: int = 64, sym: bool = False,
                     layer_policies=()):
    """Replace the selected nn.Linear modules of ``model`` by W4A16Linear / W8A16Linear
    (plain group-wise packing) following the base configuration and the policies (the
    last matching policy wins).  Returns the plan of ``plan_quantization``."""
    plan = plan_quantization(model, target_modules, bits, group_size, sym, layer_policies)
    named = dict(model.named_modules())
    for name, (b, g, s) in plan.items():
        lin = named[name]
        new = (W8A16Linear.from_weight(_weight_of(lin).contiguous(), g, None, lin.bias) if b == 8
               else W4A16Linear.from_weight(_weight_of(lin).contiguous(), g, None, lin.bias, s))
        parent_name, _, attr = name.rpartition(".")
        setattr(named[parent_name] if parent_name else model, attr, new)
    return plan
