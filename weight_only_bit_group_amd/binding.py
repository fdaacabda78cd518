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
        if name not in ("quantize", "dequantize", "gemm", "gemm_a4", "grouped_gemm", "grouped_gemm_a4"):
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
