"""Thin torch binding of libaq: the C entry points under the same names.

Argument marshalling only -- every step of the computation runs in the
library's HIP kernels.  Tensors must be CUDA (HIP) tensors; outputs are
allocated with torch when not supplied; calls are enqueued on the current
torch stream of the tensors' device.  Status 1 raises ValueError, status 2
RuntimeError, with the library's message.
"""
from __future__ import annotations

import numpy as np
import torch

from . import _lib
from ._lib import AQ_BF16, AQ_F32, check


def _stream(t: torch.Tensor) -> int:
    # raw handle of torch's current stream on the tensor's device (cheap accessor)
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _wdtype(w: torch.Tensor) -> int:
    if w.dtype == torch.float32:
        return AQ_F32
    if w.dtype == torch.bfloat16:
        return AQ_BF16
    raise ValueError(f"W must be float32 or bfloat16 (got {w.dtype})")


def _packed_outputs(w_like: torch.Tensor, n: int, k: int, group: int, packed, scales, zeros):
    dev = w_like.device
    if packed is None:
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((n, k // group), dtype=torch.float32, device=dev)
    if zeros is None:
        zeros = torch.empty((n, k // group), dtype=torch.uint8, device=dev)
    return packed, scales, zeros


def aq_quantize_pack(W: torch.Tensor, group: int, chan_scale: torch.Tensor | None = None, *,
                     packed=None, scales=None, zeros=None, sym: bool = False):
    """(packed [N, K/2] u8, scales [N, K/g] f32, zeros [N, K/g] u8) of W[N, K] (f32 or bf16).

    sym=True calls aq_quantize_pack_sym (symmetric codes, zero point 8).
    """
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, K]")
    _need(W, "W", W.dtype)
    n, k = W.shape
    if k % group:
        raise ValueError("K must be a multiple of group")
    if chan_scale is not None:
        _need(chan_scale, "chan_scale", torch.float32, 1)
    packed, scales, zeros = _packed_outputs(W, n, k, group, packed, scales, zeros)
    fn = "aq_quantize_pack_sym" if sym else "aq_quantize_pack"
    st = getattr(_lib.load(), fn)(W.data_ptr(), _wdtype(W), n, k, group, _ptr(chan_scale), packed.data_ptr(),
                                  scales.data_ptr(), zeros.data_ptr(), _stream(W))
    check(st, fn)
    return packed, scales, zeros


def _workspace(ws, need: int, device):
    """(pointer, bytes) of a workspace: allocated here when `ws` is None and `need` > 0."""
    if ws is None:
        if need <= 0:
            return None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    if ws.numel() == 0:
        return None, 0
    if ws.device.type != "cuda" or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return ws, ws.numel() * ws.element_size()


def _product(fn_name, X, packed, scales, zeros, group, out, workspace=None):
    _need(X, "X", torch.bfloat16, 2)
    _need(packed, "packed", torch.uint8, 2)
    _need(scales, "scales", torch.float32, 2)
    _need(zeros, "zeros", torch.uint8, 2)
    m, k = X.shape
    n = packed.shape[0]
    if packed.shape[1] * 2 != k:
        raise ValueError("packed must be [N, K/2] for X [M, K]")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=X.device)
    _need(out, "Y", torch.float32, 2)
    lib = _lib.load()
    if fn_name == "aq_w4a16_gemm":
        ws, nbytes = _workspace(workspace, int(lib.aq_w4a16_gemm_workspace(m, n, k, group)), X.device)
        st = lib.aq_w4a16_gemm(X.data_ptr(), m, k, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), n, group,
                               out.data_ptr(), _ptr(ws), nbytes, _stream(X))
    else:
        st = getattr(lib, fn_name)(X.data_ptr(), m, k, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                   n, group, out.data_ptr(), _stream(X))
    check(st, fn_name)
    return out


def aq_w4a16_gemv(X, packed, scales, zeros, group: int, out=None):
    """Y[M, N] fp32 = X[M, K] (bf16, 1 <= M <= 16) times the dequantized packed weight, transposed."""
    return _product("aq_w4a16_gemv", X, packed, scales, zeros, group, out)


def aq_w4a16_gemm_workspace(M: int, N: int, K: int, group: int) -> int:
    return int(_lib.load().aq_w4a16_gemm_workspace(M, N, K, group))


def aq_w4a16_gemm(X, packed, scales, zeros, group: int, out=None, workspace=None):
    """Y[M, N] fp32 = X[M, K] (bf16, any M) times the dequantized packed weight, transposed (MFMA).

    workspace: None allocates the staging matrix when the size takes the staged path;
    a uint8 device tensor is used as given (an empty one selects the fused path).
    """
    return _product("aq_w4a16_gemm", X, packed, scales, zeros, group, out, workspace)


def aq_act_absmean_workspace(T: int, K: int) -> int:
    return int(_lib.load().aq_act_absmean_workspace(T, K))


def aq_act_absmean(X, sum_abs, total_count: int, mean_out=None, workspace=None):
    """sum_abs[K] (fp64) += sum_t |X[t, K]|; mean_out[K] = fl32(sum_abs / total_count) if given."""
    _need(X, "X", torch.bfloat16, 2)
    _need(sum_abs, "sum_abs", torch.float64, 1)
    t, k = X.shape
    if mean_out is not None:
        _need(mean_out, "mean_out", torch.float32, 1)
    need = aq_act_absmean_workspace(t, k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=X.device)
    st = _lib.load().aq_act_absmean(X.data_ptr(), t, k, sum_abs.data_ptr(), _ptr(mean_out), total_count,
                                    workspace.data_ptr(), workspace.numel(), _stream(X))
    check(st, "aq_act_absmean")
    return sum_abs, mean_out


def aq_act_absmean_noalloc(X, sum_abs, total_count: int, mean_out=None):
    """aq_act_absmean with the library's own scratch (no workspace, nothing allocated)."""
    _need(X, "X", torch.bfloat16, 2)
    _need(sum_abs, "sum_abs", torch.float64, 1)
    t, k = X.shape
    if mean_out is not None:
        _need(mean_out, "mean_out", torch.float32, 1)
    st = _lib.load().aq_act_absmean_noalloc(X.data_ptr(), t, k, sum_abs.data_ptr(), _ptr(mean_out), total_count,
                                            _stream(X))
    check(st, "aq_act_absmean_noalloc")
    return sum_abs, mean_out


def aq_awq_search_workspace(T: int, N: int, K: int, group: int, n_grid: int = 20) -> int:
    return int(_lib.load().aq_awq_search_workspace(T, N, K, group, n_grid))


def aq_awq_search(X_sub, absmean_host, W, group: int, n_grid: int = 20, workspace=None):
    """Alpha-grid AWQ search.  ``absmean_host`` is a host fp32 array/tensor [K].

    Returns dict(mse [n_grid] f64, best [1] i32, best_scale [K] f32, packed, scales, zeros) on the device.
    """
    _need(X_sub, "X_sub", torch.bfloat16, 2)
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, K]")
    _need(W, "W", W.dtype)
    t, k = X_sub.shape
    n = W.shape[0]
    if W.shape[1] != k:
        raise ValueError("W must be [N, K] for X_sub [T, K]")
    m = np.ascontiguousarray(absmean_host.cpu().numpy() if isinstance(absmean_host, torch.Tensor) else absmean_host,
                             dtype=np.float32)
    if m.shape != (k,):
        raise ValueError("absmean_host must have K entries")
    dev = X_sub.device
    mse = torch.empty(n_grid, dtype=torch.float64, device=dev)
    best = torch.empty(1, dtype=torch.int32, device=dev)
    best_scale = torch.empty(k, dtype=torch.float32, device=dev)
    packed, scales, zeros = _packed_outputs(W, n, k, group, None, None, None)
    need = aq_awq_search_workspace(t, n, k, group, n_grid)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = _lib.load().aq_awq_search(X_sub.data_ptr(), t, m.ctypes.data, W.data_ptr(), _wdtype(W), n, k, group, n_grid,
                                   mse.data_ptr(), best.data_ptr(), best_scale.data_ptr(), packed.data_ptr(),
                                   scales.data_ptr(), zeros.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                   _stream(X_sub))
    check(st, "aq_awq_search")
    return {"mse": mse, "best": best, "best_scale": best_scale, "packed": packed, "scales": scales, "zeros": zeros}


def aq_awq_fold_norm(norm_w, chan_scale, out=None):
    """folded [K] fp32 = fl32(norm_w / chan_scale) on the device (norm_w fp32 or bf16; other float
    dtypes are widened to fp32 first, exactly)."""
    if norm_w.dtype not in (torch.float32, torch.bfloat16):
        norm_w = norm_w.float()
    _need(norm_w, "norm_w", norm_w.dtype, 1)
    _need(chan_scale, "chan_scale", torch.float32, 1)
    k = norm_w.shape[0]
    if chan_scale.shape[0] != k:
        raise ValueError("norm_w and chan_scale must have the same length")
    if out is None:
        out = torch.empty(k, dtype=torch.float32, device=norm_w.device)
    _need(out, "folded", torch.float32, 1)
    st = _lib.load().aq_awq_fold_norm(norm_w.data_ptr(), _wdtype(norm_w), chan_scale.data_ptr(), k, out.data_ptr(),
                                      _stream(norm_w))
    check(st, "aq_awq_fold_norm")
    return out


def aq_fp4_gemm_workspace(M: int, N: int, K: int) -> int:
    return int(_lib.load().aq_fp4_gemm_workspace(M, N, K))


def aq_fp4_gemm(X, codes, block_scales, tensor_scale: float, out=None, workspace=None):
    """Y[M, N] fp32 = tensor_scale * X[M, K] times (e2m1 * e4m3)^T for codes [N, K/2], block_scales [N, K/16]."""
    _need(X, "X", torch.bfloat16, 2)
    _need(codes, "codes", torch.uint8, 2)
    _need(block_scales, "block_scales", torch.uint8, 2)
    m, k = X.shape
    n = codes.shape[0]
    if codes.shape[1] * 2 != k or block_scales.shape != (n, k // 16):
        raise ValueError("codes must be [N, K/2] and block_scales [N, K/16]")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=X.device)
    _need(out, "Y", torch.float32, 2)
    lib = _lib.load()
    ws, nbytes = _workspace(workspace, int(lib.aq_fp4_gemm_workspace(m, n, k)), X.device)
    st = lib.aq_fp4_gemm(X.data_ptr(), m, k, codes.data_ptr(), block_scales.data_ptr(), float(tensor_scale),
                         n, out.data_ptr(), _ptr(ws), nbytes, _stream(X))
    check(st, "aq_fp4_gemm")
    return out


def aq_fp4_quantize_workspace(N: int, K: int) -> int:
    return int(_lib.load().aq_fp4_quantize_workspace(N, K))


def aq_fp4_quantize(W, *, codes=None, block_scales=None, tensor_scale=None, workspace=None):
    """(codes [N, K/2] u8, block_scales [N, K/16] u8, tensor_scale [1] f32) of W[N, K] (f32 or bf16), on the device."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, K]")
    _need(W, "W", W.dtype)
    n, k = W.shape
    if k % 16:
        raise ValueError("K must be a multiple of 16")
    dev = W.device
    if codes is None:
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
    if block_scales is None:
        block_scales = torch.empty((n, k // 16), dtype=torch.uint8, device=dev)
    if tensor_scale is None:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=dev)
    need = aq_fp4_quantize_workspace(n, k)
    if workspace is None:
        workspace = torch.empty(max(need, 4), dtype=torch.uint8, device=dev)
    st = _lib.load().aq_fp4_quantize(W.data_ptr(), _wdtype(W), n, k, codes.data_ptr(), block_scales.data_ptr(),
                                     tensor_scale.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(W))
    check(st, "aq_fp4_quantize")
    return codes, block_scales, tensor_scale


def aq_quantize_pack8(W: torch.Tensor, group: int, chan_scale: torch.Tensor | None = None, *,
                      codes=None, scales=None, zeros=None):
    """(codes [N, K] u8, scales [N, K/g] f32, zeros [N, K/g] u8) of W[N, K] (f32 or bf16), 8-bit codes."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, K]")
    _need(W, "W", W.dtype)
    n, k = W.shape
    if k % group:
        raise ValueError("K must be a multiple of group")
    if chan_scale is not None:
        _need(chan_scale, "chan_scale", torch.float32, 1)
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=W.device)
    _, scales, zeros = _packed_outputs(W, n, k, group, codes, scales, zeros)
    st = _lib.load().aq_quantize_pack8(W.data_ptr(), _wdtype(W), n, k, group, _ptr(chan_scale), codes.data_ptr(),
                                       scales.data_ptr(), zeros.data_ptr(), _stream(W))
    check(st, "aq_quantize_pack8")
    return codes, scales, zeros


def aq_w8a16_gemm_workspace(M: int, N: int, K: int, group: int) -> int:
    return int(_lib.load().aq_w8a16_gemm_workspace(M, N, K, group))


def _product8(fn_name, X, codes, scales, zeros, group, out, workspace=None):
    _need(X, "X", torch.bfloat16, 2)
    _need(codes, "codes", torch.uint8, 2)
    _need(scales, "scales", torch.float32, 2)
    _need(zeros, "zeros", torch.uint8, 2)
    m, k = X.shape
    n = codes.shape[0]
    if codes.shape[1] != k:
        raise ValueError("codes must be [N, K] for X [M, K]")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=X.device)
    _need(out, "Y", torch.float32, 2)
    lib = _lib.load()
    if fn_name == "aq_w8a16_gemm":
        need = int(lib.aq_w8a16_gemm_workspace(m, n, k, group))
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
        st = lib.aq_w8a16_gemm(X.data_ptr(), m, k, codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), n, group,
                               out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(X))
    else:
        st = lib.aq_w8a16_gemv(X.data_ptr(), m, k, codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), n, group,
                               out.data_ptr(), _stream(X))
    check(st, fn_name)
    return out


def aq_w8a16_gemv(X, codes, scales, zeros, group: int, out=None):
    """Y[M, N] fp32 = X[M, K] (bf16, 1 <= M <= 16) times the dequantized 8-bit weight, transposed."""
    return _product8("aq_w8a16_gemv", X, codes, scales, zeros, group, out)


def aq_w8a16_gemm(X, codes, scales, zeros, group: int, out=None, workspace=None):
    """Y[M, N] fp32 = X[M, K] (bf16, any M) times the dequantized 8-bit weight (staged bf16 + MFMA)."""
    return _product8("aq_w8a16_gemm", X, codes, scales, zeros, group, out, workspace)


# ---- MXFP4 -------------------------------------------------------------------------------
# These calls also run on a device that is not the current one (every tensor has to be on
# X's device), and X may have rows further apart than their length.  A call on a few rows is
# a matter of microseconds on the host, so the module _aq_torch makes the common call whole;
# where it returns None (a wrong argument, another device, an empty product, an error) the call
# is gone through here.


class _MxNative:
    """The module's functions; the first use of one loads the library and the module."""

    def __getattr__(self, name):
        if name not in ("quantize", "dequantize", "gemm", "gemm_a4", "grouped_gemm", "grouped_gemm_a4", "fp8_quantize",
                        "fp8_dequantize", "fp8_gemm", "fp8_grouped_gemm", "fp8_linear", "fp8_experts", "route",
                        "route_graph", "capture_conflict", "route_backward"):
            raise AttributeError(name)
        _lib.load()
        from . import _aq_torch   # an ImportError here: the module has not been built
        fn = getattr(_aq_torch, name)
        setattr(self, name, fn)
        return fn


_mx = _MxNative()


def _mx_call(name: str, dev: int, *args) -> None:
    fn = getattr(_lib.load(), name)
    with torch.cuda.device(dev):
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    check(st, name)


def _mx_need(t, name: str, dtype, shape, dev: int):
    """Raises unless t is a dense GPU tensor of this type and shape on device dev."""
    _need(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev} (got {t.device})")


def _mx_rows(X, name: str, types):
    """(rows, columns, row stride in elements, device) of a GPU matrix whose rows are dense."""
    if not isinstance(X, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not X.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got {X.device})")
    if X.dtype not in types:
        raise ValueError(f"{name} must be {' or '.join(str(t) for t in types)} (got {X.dtype})")
    if X.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions")
    m, k = X.shape
    if k == 0 or k & 31:
        raise ValueError(f"K must be a positive multiple of 32 (got {k})")
    ld = k
    if not X.is_contiguous():
        ld, step = X.stride()
        if m <= 1:   # (the stride of a single row says nothing)
            ld = k
        if step != 1 or ld < k:
            raise ValueError(f"{name} must have dense rows (strides {X.stride()})")
    return m, k, ld, X.get_device()


_U8 = torch.uint8


def _mx_codes(codes, scales, name: str, scales_name: str):
    """(rows, columns, device) of an MXFP4 matrix: codes [M, K/2], scales [M, K/32]."""
    _need(codes, name, _U8, 2)
    m, half = codes.shape
    if half == 0 or half & 15:
        raise ValueError(f"K must be a positive multiple of 32 (got {2 * half})")
    dev = codes.get_device()
    _mx_need(scales, scales_name, _U8, (m, half >> 4), dev)
    return m, 2 * half, dev


def _mx_weights(codes, scales, k: int, dev: int, ndim: int):
    """The shape (N,) or (E, N) of MXFP4 weights with rows of k."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != ndim:
        raise ValueError("codes must be [N, K/2]" if ndim == 2 else "codes must be [E, N, K/2]")
    lead = codes.shape[:-1]
    _mx_need(codes, "codes", _U8, (*lead, k // 2), dev)
    _mx_need(scales, "scales", _U8, (*lead, k >> 5), dev)
    return lead


_MX_OUT = {torch.float32: AQ_F32, torch.bfloat16: AQ_BF16}


def _mx_out(out, m: int, n: int, out_dtype, like, dev: int):
    """(the output tensor, its dtype code); out gives the type when out_dtype is None."""
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    code = _MX_OUT.get(out_dtype)
    if code is None:
        raise ValueError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
    if out is None:
        return like.new_empty((m, n), dtype=out_dtype), code
    _mx_need(out, "Y", out_dtype, (m, n), dev)
    return out, code


def aq_mxfp4_quantize(X, *, codes=None, scales=None):
    """(codes [M, K/2] u8, scales [M, K/32] u8) of X[M, K] (f32 or bf16; its rows may be strided)."""
    if codes is None and scales is None:
        pair = _mx.quantize(X)
        if pair is not None:
            return pair
    m, k, ld, dev = _mx_rows(X, "X", _MX_OUT)
    if codes is None:
        codes = X.new_empty((m, k >> 1), dtype=torch.uint8)
    else:
        _mx_need(codes, "codes", torch.uint8, (m, k >> 1), dev)
    if scales is None:
        scales = X.new_empty((m, k >> 5), dtype=torch.uint8)
    else:
        _mx_need(scales, "scales", torch.uint8, (m, k >> 5), dev)
    if m:
        _mx_call("aq_mxfp4_quantize", dev, X.data_ptr(), _MX_OUT[X.dtype], m, k, ld, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def aq_mxfp4_dequantize(codes, scales, out_dtype=None, out=None):
    """Y[M, K] (float32, or bfloat16: exact in both) = the values of codes [M, K/2] and scales [M, K/32]."""
    y = _mx.dequantize(codes, scales, out_dtype, out)
    if y is not None:
        return y
    m, k, dev = _mx_codes(codes, scales, "codes", "scales")
    out, code = _mx_out(out, m, k, out_dtype, codes, dev)
    if m:
        _mx_call("aq_mxfp4_dequantize", dev, codes.data_ptr(), scales.data_ptr(), m, k, out.data_ptr(), code)
    return out


def aq_mxfp4_gemm(X, codes, scales, out_dtype=None, out=None):
    """Y[M, N] (float32, or bfloat16) = X[M, K] (bf16; its rows may be strided) times the MXFP4 weights, transposed."""
    y = _mx.gemm(X, codes, scales, out_dtype, out)
    if y is not None:
        return y
    m, k, ld, dev = _mx_rows(X, "X", (torch.bfloat16,))
    n, = _mx_weights(codes, scales, k, dev, 2)
    out, code = _mx_out(out, m, n, out_dtype, X, dev)
    if m and n:
        _mx_call("aq_mxfp4_gemm", dev, X.data_ptr(), m, k, ld, codes.data_ptr(), scales.data_ptr(), n, out.data_ptr(), code)
    return out


def aq_mxfp4_gemm_a4(X_codes, X_scales, codes, scales, out_dtype=None, out=None):
    """Y[M, N] (float32, or bfloat16) of MXFP4 activations (as aq_mxfp4_quantize returns them) and MXFP4 weights."""
    y = _mx.gemm_a4(X_codes, X_scales, codes, scales, out_dtype, out)
    if y is not None:
        return y
    m, k, dev = _mx_codes(X_codes, X_scales, "X_codes", "X_scales")
    n, = _mx_weights(codes, scales, k, dev, 2)
    out, code = _mx_out(out, m, n, out_dtype, X_codes, dev)
    if m and n:
        _mx_call("aq_mxfp4_gemm_a4", dev, X_codes.data_ptr(), X_scales.data_ptr(), m, k, codes.data_ptr(),
                 scales.data_ptr(), n, out.data_ptr(), code)
    return out


def _mx_lists(offsets, rows, e: int, t: int, dev: int) -> int:
    """Rows of Y: the length of rows, or all t rows of X."""
    _mx_need(offsets, "offsets", torch.int32, (e + 1,), dev)
    if rows is None:
        return t
    _need(rows, "rows", torch.int32, 1)
    if rows.get_device() != dev:
        raise ValueError(f"rows must be on cuda:{dev} (got {rows.device})")
    return rows.shape[0]


def aq_mxfp4_grouped_gemm(X, codes, scales, offsets, rows=None, out_dtype=None, out=None):
    """Y[M, N]: rows offsets[e] .. offsets[e + 1] - 1 are X's rows (or those that ``rows`` [M] lists) times expert
    e's MXFP4 weights, transposed.

    X [T, K] bf16 (its rows may be strided), codes [E, N, K/2], scales [E, N, K/32], offsets [E + 1] int32 and rows
    int32 on the device.  Rows of Y outside the offsets are not written.
    """
    y = _mx.grouped_gemm(X, codes, scales, offsets, rows, out_dtype, out)
    if y is not None:
        return y
    t, k, ld, dev = _mx_rows(X, "X", (torch.bfloat16,))
    e, n = _mx_weights(codes, scales, k, dev, 3)
    m = _mx_lists(offsets, rows, e, t, dev)
    out, code = _mx_out(out, m, n, out_dtype, X, dev)
    if m and n:
        _mx_call("aq_mxfp4_grouped_gemm", dev, X.data_ptr(), t, k, ld, codes.data_ptr(), scales.data_ptr(), e, n,
                 offsets.data_ptr(), None if rows is None else rows.data_ptr(), m, out.data_ptr(), code)
    return out


def aq_mxfp4_grouped_gemm_a4(X_codes, X_scales, codes, scales, offsets, rows=None, out_dtype=None, out=None):
    """aq_mxfp4_grouped_gemm with the activations in MXFP4 (X_codes [T, K/2], X_scales [T, K/32])."""
    y = _mx.grouped_gemm_a4(X_codes, X_scales, codes, scales, offsets, rows, out_dtype, out)
    if y is not None:
        return y
    t, k, dev = _mx_codes(X_codes, X_scales, "X_codes", "X_scales")
    e, n = _mx_weights(codes, scales, k, dev, 3)
    m = _mx_lists(offsets, rows, e, t, dev)
    out, code = _mx_out(out, m, n, out_dtype, X_codes, dev)
    if m and n:
        _mx_call("aq_mxfp4_grouped_gemm_a4", dev, X_codes.data_ptr(), X_scales.data_ptr(), t, k, codes.data_ptr(),
                 scales.data_ptr(), e, n, offsets.data_ptr(), None if rows is None else rows.data_ptr(), m,
                 out.data_ptr(), code)
    return out


# ---- FP8 (E4M3, a scale for each block of 128) ---------------------------------------------
# As the MXFP4 calls these run on the device of their tensors, and the common call through _aq_torch.  Codes are float8_e4m3fn; uint8
# tensors of the same bytes are taken too.

_F8 = torch.float8_e4m3fn


def _f8_codes(t, name: str, shape, dev: int) -> None:
    """Raises unless t holds dense FP8 codes of this shape on device dev."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    _mx_need(t, name, _U8 if t.dtype == _U8 else _F8, shape, dev)


def _f8_matrix(X, name: str, types):
    """(shape [.., N, K], E, N, K, row stride, device) of a matrix or a stack of them whose rows are dense."""
    if not isinstance(X, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not X.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got {X.device})")
    if X.dtype not in types:
        raise ValueError(f"{name} must be {' or '.join(str(t) for t in types)} (got {X.dtype})")
    if X.dim() not in (2, 3):
        raise ValueError(f"{name} must have 2 or 3 dimensions")
    n, k = X.shape[-2:]
    e = X.shape[0] if X.dim() == 3 else 1
    if k == 0 or k % 16:
        raise ValueError(f"K must be a positive multiple of 16 (got {k})")
    ld = k
    if not X.is_contiguous() and X.numel():
        ld = X.stride(-2) if n > 1 else X.stride(0) if e > 1 and X.dim() == 3 else k
        if X.stride(-1) != 1 or ld < k or (e > 1 and X.stride(0) != n * ld):
            raise ValueError(f"{name} must have dense rows, evenly spaced (strides {X.stride()})")
    return tuple(X.shape), e, n, k, ld, X.get_device()


def _f8_scales(shape, block_rows: int):
    """The shape of the scales of codes [.., N, K]."""
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128 (got {block_rows})")
    return (*shape[:-2], -(-shape[-2] // block_rows), -(-shape[-1] // 128))


def aq_fp8_quantize(X, block_rows: int = 1, *, codes=None, scales=None):
    """(codes [.., N, K] float8_e4m3fn, scales f32) of X [N, K] or [E, N, K] (f32 or bf16; its rows may be strided).

    block_rows=1: a scale for 128 k of each row, scales [.., N, ceil(K / 128)] (activations);
    block_rows=128: for 128 rows by 128 k, scales [.., ceil(N / 128), ceil(K / 128)] (weights).
    """
    if codes is None and scales is None:
        pair = _mx.fp8_quantize(X, block_rows)
        if pair is not None:
            return pair
    shape, e, n, k, ld, dev = _f8_matrix(X, "X", _MX_OUT)
    sshape = _f8_scales(shape, block_rows)
    if codes is None:
        codes = X.new_empty(shape, dtype=_F8)
    else:
        _f8_codes(codes, "codes", shape, dev)
    if scales is None:
        scales = X.new_empty(sshape, dtype=torch.float32)
    else:
        _mx_need(scales, "scales", torch.float32, sshape, dev)
    if e and n:
        _mx_call("aq_fp8_quantize", dev, X.data_ptr(), _MX_OUT[X.dtype], e, n, k, ld, block_rows, codes.data_ptr(),
                 scales.data_ptr())
    return codes, scales


def aq_fp8_dequantize(codes, scales, block_rows: int = 1, out_dtype=None, out=None):
    """Y [.., N, K] (float32, or bfloat16) = the values of codes [.., N, K] and their scales (as aq_fp8_quantize)."""
    y = _mx.fp8_dequantize(codes, scales, block_rows, out_dtype, out)
    if y is not None:
        return y
    shape, e, n, k, _, dev = _f8_matrix(codes, "codes", (_F8, _U8))
    _f8_codes(codes, "codes", shape, dev)
    _mx_need(scales, "scales", torch.float32, _f8_scales(shape, block_rows), dev)
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    code = _MX_OUT.get(out_dtype)
    if code is None:
        raise ValueError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
    if out is None:
        out = codes.new_empty(shape, dtype=out_dtype)
    else:
        _mx_need(out, "Y", out_dtype, shape, dev)
    if e and n:
        _mx_call("aq_fp8_dequantize", dev, codes.data_ptr(), scales.data_ptr(), e, n, k, block_rows, out.data_ptr(), code)
    return out


def _f8_rows(codes, scales):
    """(rows, columns, device) of FP8 activations: codes [M, K], scales [M, ceil(K / 128)]."""
    if getattr(codes, "ndim", 2) != 2:
        raise ValueError("X_codes must have 2 dimensions")
    (m, k), *_, dev = _f8_matrix(codes, "X_codes", (_F8, _U8))
    _f8_codes(codes, "X_codes", (m, k), dev)
    _mx_need(scales, "X_scales", torch.float32, (m, -(-k // 128)), dev)
    return m, k, dev


def _f8_weights(codes, scales, k: int, dev: int, ndim: int):
    """The shape (N,) or (E, N) of FP8 weights with rows of k."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != ndim:
        raise ValueError("codes must be [N, K]" if ndim == 2 else "codes must be [E, N, K]")
    lead = codes.shape[:-1]
    _f8_codes(codes, "codes", (*lead, k), dev)
    _mx_need(scales, "scales", torch.float32, _f8_scales((*lead, k), 128), dev)
    return lead


def aq_fp8_gemm(X_codes, X_scales, codes, scales, out_dtype=None, out=None):
    """Y[M, N] (float32, or bfloat16) of FP8 activations (as aq_fp8_quantize returns them) and FP8 weights, transposed.

    codes [N, K], scales [ceil(N / 128), ceil(K / 128)] (as aq_fp8_quantize with block_rows=128 returns them).
    """
    y = _mx.fp8_gemm(X_codes, X_scales, codes, scales, out_dtype, out)
    if y is not None:
        return y
    m, k, dev = _f8_rows(X_codes, X_scales)
    n, = _f8_weights(codes, scales, k, dev, 2)
    out, code = _mx_out(out, m, n, out_dtype, X_codes, dev)
    if m and n:
        _mx_call("aq_fp8_gemm", dev, X_codes.data_ptr(), X_scales.data_ptr(), m, k, codes.data_ptr(), scales.data_ptr(), n,
                 out.data_ptr(), code)
    return out


def _f8_values(X):
    """(rows, columns, row stride, device) of the activations X [M, K]."""
    if getattr(X, "ndim", 2) != 2:
        raise ValueError("X must have 2 dimensions")
    (m, k), _, _, _, ld, dev = _f8_matrix(X, "X", _MX_OUT)
    return m, k, ld, dev


def _f8_workspace(workspace, need: int, like, dev: int):
    if workspace is None:
        return like.new_empty(need, dtype=_U8)
    _need(workspace, "workspace", _U8, 1)
    if workspace.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev} (got {workspace.device})")
    return workspace


def aq_fp8_linear_workspace(M: int, K: int) -> int:
    return int(_lib.load().aq_fp8_linear_workspace(M, K))


def aq_fp8_linear(X, codes, scales, out_dtype=None, out=None, workspace=None):
    """Y[M, N] (float32, or bfloat16) = X[M, K] (f32 or bf16, rounded to FP8 on the way; its rows may be strided) times
    the FP8 weights, transposed.

    workspace: None allocates it; a uint8 device tensor is used as given.
    """
    if workspace is None:
        y = _mx.fp8_linear(X, codes, scales, out_dtype, out)
        if y is not None:
            return y
    m, k, ld, dev = _f8_values(X)
    n, = _f8_weights(codes, scales, k, dev, 2)
    out, code = _mx_out(out, m, n, out_dtype, X, dev)
    if m and n:
        workspace = _f8_workspace(workspace, aq_fp8_linear_workspace(m, k), X, dev)
        _mx_call("aq_fp8_linear", dev, X.data_ptr(), _MX_OUT[X.dtype], m, k, ld, codes.data_ptr(), scales.data_ptr(), n,
                 out.data_ptr(), code, workspace.data_ptr(), workspace.numel())
    return out


def aq_fp8_grouped_gemm(X_codes, X_scales, codes, scales, offsets, rows=None, out_dtype=None, out=None):
    """Y[M, N]: rows offsets[e] .. offsets[e + 1] - 1 are X's rows (or those that ``rows`` [M] lists) times expert
    e's FP8 weights, transposed.

    X_codes [T, K], X_scales [T, ceil(K / 128)], codes [E, N, K], scales [E, ceil(N / 128), ceil(K / 128)], offsets
    [E + 1] int32 and rows int32 on the device.  Rows of Y outside the offsets are not written.
    """
    y = _mx.fp8_grouped_gemm(X_codes, X_scales, codes, scales, offsets, rows, out_dtype, out)
    if y is not None:
        return y
    t, k, dev = _f8_rows(X_codes, X_scales)
    e, n = _f8_weights(codes, scales, k, dev, 3)
    m = _mx_lists(offsets, rows, e, t, dev)
    out, code = _mx_out(out, m, n, out_dtype, X_codes, dev)
    if m and n:
        _mx_call("aq_fp8_grouped_gemm", dev, X_codes.data_ptr(), X_scales.data_ptr(), t, k, codes.data_ptr(),
                 scales.data_ptr(), e, n, offsets.data_ptr(), None if rows is None else rows.data_ptr(), m, out.data_ptr(),
                 code)
    return out


def aq_fp8_swiglu_quantize(H, end=None, *, codes=None, scales=None):
    """(codes [M, I] float8_e4m3fn, scales [M, ceil(I / 128)] f32) of silu(g) * u for rows [g | u] of H [M, 2 I] (f32 or
    bf16); end: rows from this device count (int32 [1]) on are left out."""
    if getattr(H, "ndim", 2) != 2:
        raise ValueError("H must have 2 dimensions")
    (m, k), *_, dev = _f8_matrix(H, "H", _MX_OUT)
    _need(H, "H", H.dtype)
    if k % 32:
        raise ValueError(f"H must be [M, 2 I] with I a multiple of 16 (got {list(H.shape)})")
    shape = (m, k // 2)
    if end is not None:
        _mx_need(end, "end", torch.int32, (1,), dev)
    if codes is None:
        codes = H.new_empty(shape, dtype=_F8)
    else:
        _f8_codes(codes, "codes", shape, dev)
    if scales is None:
        scales = H.new_empty(_f8_scales(shape, 1), dtype=torch.float32)
    else:
        _mx_need(scales, "scales", torch.float32, _f8_scales(shape, 1), dev)
    if m:
        _mx_call("aq_fp8_swiglu_quantize", dev, H.data_ptr(), _MX_OUT[H.dtype], m, k // 2, _ptr(end), codes.data_ptr(),
                 scales.data_ptr())
    return codes, scales


def aq_fp8_experts_workspace(T: int, top: int, K: int, E: int, I: int) -> int:
    return int(_lib.load().aq_fp8_experts_workspace(T, top, K, E, I))


def aq_fp8_experts(X, gate_up_codes, gate_up_scales, down_codes, down_scales, ids, weights, out_dtype=None, workspace=None):
    """(out [T, K], products [T * top, K] f32, slots [T, top] int32): a mixture's gated experts with FP8 weights.

    out[t] = sum_j weights[t, j] D_e Q(silu(G_e Q(x[t])) * U_e Q(x[t])) for the experts e = ids[t, j] (int32; others than
    0 .. E - 1 add nothing), Q the rounding to FP8 rows.  gate_up [E, 2I, K] and down [E, K, I] as codes and scales in
    128 x 128 blocks; X f32 or bf16, its rows may be strided; weights f32; out float32, or bfloat16 with the second
    product on the FP8 matrix instructions.  products holds a choice's result in row slots[t, j] (not written for a choice
    without an expert), as aq_moe_combine and its gradient take them.
    workspace: None allocates it; a uint8 device tensor is used as given.
    """
    if workspace is None:
        got = _mx.fp8_experts(X, gate_up_codes, gate_up_scales, down_codes, down_scales, ids, weights, out_dtype)
        if got is not None:
            return got
    t, k, ld, dev = _f8_values(X)
    e, n = _f8_weights(gate_up_codes, gate_up_scales, k, dev, 3)
    if n % 2:
        raise ValueError(f"gate_up must be [E, 2I, K] (got {[e, n, k]})")
    if tuple(_f8_weights(down_codes, down_scales, n // 2, dev, 3)) != (e, k):
        raise ValueError(f"down must be {[e, k, n // 2]} (got {list(down_codes.shape)})")
    _need(ids, "ids", torch.int32, 2)
    top = ids.shape[1]
    _mx_need(ids, "ids", torch.int32, (t, top), dev)
    _mx_need(weights, "weights", torch.float32, (t, top), dev)
    out, code = _mx_out(None, t, k, out_dtype, X, dev)
    products, slots = X.new_empty((t * top, k), dtype=torch.float32), torch.empty_like(ids)
    workspace = _f8_workspace(workspace, aq_fp8_experts_workspace(t, top, k, e, n // 2), X, dev)
    _mx_call("aq_fp8_experts", dev, X.data_ptr(), _MX_OUT[X.dtype], t, k, ld, gate_up_codes.data_ptr(),
             gate_up_scales.data_ptr(), down_codes.data_ptr(), down_scales.data_ptr(), e, n // 2, ids.data_ptr(),
             weights.data_ptr(), top, products.data_ptr(), slots.data_ptr(), out.data_ptr(), code, workspace.data_ptr(),
             workspace.numel())
    return out, products, slots


# ---- routing to experts --------------------------------------------------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}


def _logits(logits):
    """(T, E, row stride, device) of router logits [T, E] whose rows are dense."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError(f"logits must be a GPU tensor (got {logits.device})")
    if logits.dtype not in _MX_OUT:
        raise ValueError(f"logits must be float32 or bfloat16 (got {logits.dtype})")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    t, e = logits.shape
    ld = logits.stride(0) if t > 1 else e
    if t and e and (logits.stride(1) != 1 and e > 1 or ld < e):
        raise ValueError(f"logits must have dense rows (strides {logits.stride()})")
    return t, e, ld, logits.get_device()


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid' (got {score!r})")
    return _SCORES[score]


def aq_moe_route(logits, top: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: int | None = None,
                 renormalize: bool = True, scale: float = 1.0):
    """(ids [T, top] int32, weights [T, top] f32) of router logits [T, E] (f32 or bf16; rows may be strided).

    score: "softmax" or "sigmoid"; bias [E] f32 is added to the scores for the choice alone; groups > 1 keeps the
    experts of the top_groups best runs of E / groups neighbours, a run's score being the sum of its two highest (scores
    plus bias) whether or not there is a bias, never its highest alone; renormalize divides a token's weights by their sum.
    An expert whose logit is -inf is never chosen; slots left over get id -1 and weight 0.
    """
    pair = _mx.route(logits, top, score, bias, groups, top_groups, renormalize, scale)
    if pair is not None:
        return pair
    t, e, ld, dev = _logits(logits)
    if bias is not None:
        _mx_need(bias, "bias", torch.float32, (e,), dev)
    if not 0 < top <= min(e, 64):
        raise ValueError(f"top must be 1 .. 64 and at most E (got {top} of {e})")
    top_groups = groups if top_groups is None else top_groups
    if not 0 < top_groups <= groups <= 64:   # (ctypes would cut them down to 32 bits)
        raise ValueError(f"groups must be 1 .. 64 and top_groups 1 .. groups (got {groups} and {top_groups})")
    ids = logits.new_empty((t, top), dtype=torch.int32)
    weights = logits.new_empty((t, top), dtype=torch.float32)
    _mx_call("aq_moe_route", dev, logits.data_ptr() or 16, _MX_OUT[logits.dtype], t, e, ld, top, _score(score), _ptr(bias),
             groups, top_groups, int(bool(renormalize)), float(scale), ids.data_ptr() or 16,
             weights.data_ptr() or 16)
    return ids, weights


def moe_route_graph(logits, top: int, bias, score: str, groups: int, top_groups, renormalize: bool, scale: float):
    """aq_moe_route's result, the weights part of the graph where the logits are, or None where the native module does
    not make the call."""
    return _mx.route_graph(logits, top, score, bias, groups, top_groups, renormalize, scale)


def capture_conflict(t) -> bool:
    """Whether the current stream is being captured and t's graph reaches a leaf that a graph of an earlier call, on another
    stream, holds: the backward pass could not be captured."""
    return bool(_mx.capture_conflict(t))


def aq_moe_route_backward(logits, ids, weights, dweights, *, score: str = "softmax", renormalize: bool = True,
                          scale: float = 1.0):
    """dlogits [T, E] (the logits' type): the gradient of sum(dweights * weights) at the choices that aq_moe_route made."""
    y = _mx.route_backward(logits, ids, weights, dweights, score, renormalize, scale)
    if y is not None:
        return y
    t, e, ld, dev = _logits(logits)
    if getattr(ids, "ndim", 0) != 2:
        raise ValueError("ids must be [T, top]")
    shape = (t, ids.shape[1])
    _mx_need(ids, "ids", torch.int32, shape, dev)
    _mx_need(weights, "weights", torch.float32, shape, dev)
    _mx_need(dweights, "dweights", torch.float32, shape, dev)
    dlogits = torch.empty((t, e), dtype=logits.dtype, device=logits.device)
    if t:
        _mx_call("aq_moe_route_backward", dev, logits.data_ptr(), _MX_OUT[logits.dtype], t, e, ld, shape[1], _score(score),
                 int(bool(renormalize)), float(scale), ids.data_ptr(), weights.data_ptr(), dweights.data_ptr(), dlogits.data_ptr())
    return dlogits


def aq_moe_group_workspace(T: int, top: int, E: int) -> int:
    return int(_lib.load().aq_moe_group_workspace(T, top, E))


def aq_moe_group(ids, E: int, workspace=None):
    """(offsets [E + 1], rows [T * top], slots [T, top]), int32: choices ids [T, top] (int32) grouped by expert.

    Expert e's choices take the slots offsets[e] .. offsets[e + 1] - 1 in the order of their tokens; rows gives each
    slot's token, slots each choice's slot, -1 for an id outside 0 .. E - 1.  rows[offsets[E]:] is not written.
    """
    _need(ids, "ids", torch.int32, 2)
    t, top = ids.shape
    dev = ids.get_device()
    if not 0 < E <= 1024 or top == 0:
        raise ValueError(f"ids must be [T, top] of 1 .. 1024 experts (got {list(ids.shape)}, E {E})")
    offsets, rows, slots = ids.new_empty(E + 1), ids.new_empty(t * top), torch.empty_like(ids)
    if workspace is None:
        need = aq_moe_group_workspace(t, top, E)
        workspace = ids.new_empty(need, dtype=_U8) if need else None
    else:
        _need(workspace, "workspace", _U8, 1)
        if workspace.get_device() != dev:
            raise ValueError(f"workspace must be on cuda:{dev} (got {workspace.device})")
    # (an empty tensor has no address; nothing is read there)
    _mx_call("aq_moe_group", dev, ids.data_ptr() or 16, t, top, E, offsets.data_ptr(), rows.data_ptr() or 16,
             slots.data_ptr() or 16, _ptr(workspace), 0 if workspace is None else workspace.numel())
    return offsets, rows, slots


def _combine_args(Y, slots):
    _need(Y, "Y", Y.dtype if isinstance(Y, torch.Tensor) and Y.dtype in _MX_OUT else torch.float32, 2)
    dev = Y.get_device()
    _need(slots, "slots", torch.int32, 2)
    _mx_need(slots, "slots", torch.int32, slots.shape, dev)
    return *Y.shape, *slots.shape, dev


def aq_moe_combine(Y, slots, weights, out_dtype=None, out=None):
    """out [T, K] (float32, or bfloat16) = sum_j weights[t, j] Y[slots[t, j]] of Y [R, K] (f32 or bf16), slots [T, top]
    int32 (outside 0 .. R - 1: adds nothing) and weights [T, top] f32."""
    r, k, t, top, dev = _combine_args(Y, slots)
    _mx_need(weights, "weights", torch.float32, (t, top), dev)
    out, code = _mx_out(out, t, k, out_dtype, Y, dev)
    if t and k:
        _mx_call("aq_moe_combine", dev, Y.data_ptr() or 16, _MX_OUT[Y.dtype], r, k, slots.data_ptr(), weights.data_ptr(), t, top,
                 out.data_ptr(), code)
    return out


def aq_moe_combine_backward(Y, slots, dout):
    """dweights [T, top] f32 = sum_k dout[t, k] Y[slots[t, j], k]; 0 for a slot outside 0 .. R - 1."""
    r, k, t, top, dev = _combine_args(Y, slots)
    _mx_need(dout, "dout", dout.dtype if getattr(dout, "dtype", None) in _MX_OUT else torch.float32, (t, k), dev)
    dweights = torch.zeros((t, top), dtype=torch.float32, device=Y.device) if k == 0 else Y.new_empty((t, top), dtype=torch.float32)
    if t and k:
        _mx_call("aq_moe_combine_backward", dev, Y.data_ptr() or 16, _MX_OUT[Y.dtype], r, k, slots.data_ptr(), t, top,
                 dout.data_ptr(), _MX_OUT[dout.dtype], dweights.data_ptr())
    return dweights
