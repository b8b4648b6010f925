"""Python binding of libsq (include/sq.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch CUDA
tensors (bf16 matrices as ``torch.bfloat16``, codes as ``torch.int8``, scales as
``torch.float32``); it checks dtypes, shapes and strides, passes raw device
pointers and the current (or given) stream, and raises ``SqError`` on a non-OK
status. All computation happens in the library's CUDA kernels; there is no
fallback of any kind: if ``libsq.so`` is missing, importing this module fails.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
# SQ_LIB_PATH selects another build of the same ABI (the bounds-guard build libsq_debug.so)
LIB_PATH = os.environ.get("SQ_LIB_PATH") or os.path.join(_HERE, "libsq.so")

SQ_OK, SQ_ERR_INVALID, SQ_ERR_ALIGN, SQ_ERR_CUDA, SQ_ERR_TIMEOUT, SQ_ERR_WORKSPACE, SQ_ERR_UNSUPPORTED = \
    0, -1, -2, -3, -4, -5, -6
SQ_ERR_BOUNDS = -7
SQ_PER_TENSOR, SQ_PER_CHANNEL = 0, 1
SQ_OP_SMOOTH_QUANT_WEIGHT, SQ_OP_INT8_GEMM_DEQUANT, SQ_OP_LLMINT8 = 1, 2, 3
SQ_OP_QUANT_ACT_PER_TENSOR, SQ_OP_MEAN_STD_THRESHOLD, SQ_OP_ABS_PERCENTILE = 4, 5, 6
SQ_OP_PAGED_ATTENTION = 7
SQ_NORM_LAYER, SQ_NORM_RMS = 0, 1
SQ_KV_BF16, SQ_KV_INT8 = 0, 1

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m w8a8_quantized_gemm_b200.build`")

_lib = C.CDLL(LIB_PATH)
_p, _i64, _i32, _f32, _sz = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_size_t
_SIGS = {
    "sq_act_channel_absmax": ([_p, _i64, _i64, _i64, _p, _i32, _p], _i32),
    "sq_smooth_scale": ([_p, _p, _i64, _i64, _i64, _f32, _p, _p, _p], _i32),
    "sq_smooth_quant_weight": ([_p, _i64, _i64, _i64, _p, _i32, _p, _p, _p, _sz, _p], _i32),
    "sq_quant_act_per_token": ([_p, _i64, _i64, _i64, _p, _p, _p, _p], _i32),
    "sq_int8_gemm_dequant": ([_p, _p, _p, _p, _i32, _p, _p, _i64, _i64, _i64, _p, _p, _sz, _p], _i32),
    "llmint8_decomposed_linear": ([_p, _p, _p, _p, _f32, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _sz, _p], _i32),
    "sq_smooth_quant_weight_noalloc": ([_p, _i64, _i64, _i64, _p, _i32, _p, _p, _p], _i32),
    "sq_quant_act_per_tensor": ([_p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _sz, _p], _i32),
    "sq_smooth_scale_ex": ([_p, _p, _i64, _i64, _i64, _f32, _i32, _p, _p, _p], _i32),
    "sq_int8_gemm_dequant_ex": ([_p, _p, _p, _i32, _p, _p, _i32, _p, _p, _p, _i64, _i64, _i64, _p, _p, _sz, _p],
                                _i32),
    "sq_norm_smooth_quant": ([_p, _i64, _i64, _i64, _i32, _p, _p, _f32, _p, _p, _p, _p, _p], _i32),
    "sq_act_mean_std_threshold": ([_p, _i64, _i64, _i64, C.c_double, _p, _p, _p, _sz, _p], _i32),
    "llmint8_decomposed_linear_ex": ([_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _sz, _p], _i32),
    "sq_act_abs_percentile": ([_p, _i64, _i64, _i64, C.c_double, _p, _p, _sz, _p], _i32),
    "sq_quant_act_per_token_asym": ([_p, _i64, _i64, _i64, _p, _p, _p, _p, _p], _i32),
    "sq_weight_row_sums": ([_p, _i64, _i64, _p, _p], _i32),
    "sq_int4_weight_bytes": ([_i64, _i64], _sz),
    "sq_quant_weight_int4": ([_p, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _p], _i32),
    "sq_dequant_weight_int4": ([_p, _p, _p, _i64, _i64, _i64, _p, _p], _i32),
    "sq_int4_linear": ([_p, _i64, _i64, _i64, _p, _p, _p, _i64, _p, _p, _i64, _p], _i32),
    "sq_rope_kv_append": ([_p, _i64, _p, _i64, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _i32, _p, _p, _p, _p, _p],
                          _i32),
    "sq_paged_attention": ([_p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _i64, _f32, _p, _p, _p, _sz, _p], _i32),
    "sq_workspace_size": ([_i32, _i64, _i64, _i64], _sz),
    "sq_last_error": ([], C.c_char_p),
    "sq_sync_status": ([_p], _i32),
    "sq_version": ([], C.c_char_p),
    "sq_debug_arm_fault": ([_i32, C.c_uint64], None),
    "sq_debug_guard_margin": ([_i64], _i32),
    "sq_debug_gemm_plan": ([_i64, _i64, _i64, _i32, _p], _i32),
    "sq_kernel_launch_count": ([], C.c_uint64),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class SqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


def lib():
    """The loaded ctypes library (raw C entry points)."""
    return _lib


def sq_last_error() -> str:
    return (_lib.sq_last_error() or b"").decode()


def sq_version() -> str:
    return _lib.sq_version().decode()


def _check(st: int):
    if st != SQ_OK:
        raise SqError(st, sq_last_error())


def _torch():
    import torch
    return torch


def _stream(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t, dtype=None, name="tensor", rowmajor=False):
    if t is None:
        return None
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if rowmajor:
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} must be 2-D with unit column stride")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _ws(ws):
    if ws is None:
        return None, 0
    return _ptr(ws, None, "ws"), ws.numel() * ws.element_size()


def sq_act_channel_absmax(X, amax, accumulate: bool = False, stream=None):
    torch = _torch()
    M, K = X.shape
    _check(_lib.sq_act_channel_absmax(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0),
                                      _ptr(amax, torch.float32, "amax"), int(bool(accumulate)), _stream(stream)))
    return amax


def sq_smooth_scale(act_amax, W, alpha: float, s, inv_s, stream=None):
    torch = _torch()
    N, K = W.shape
    _check(_lib.sq_smooth_scale(_ptr(act_amax, torch.float32, "act_amax"), _ptr(W, torch.bfloat16, "W", True), N, K,
                                W.stride(0), float(alpha), _ptr(s, torch.float32, "s"),
                                _ptr(inv_s, torch.float32, "inv_s"), _stream(stream)))
    return s, inv_s


def sq_smooth_quant_weight(W, s, gran: int, Wq, w_scale, ws=None, stream=None):
    torch = _torch()
    N, K = W.shape
    wsp, wsb = _ws(ws)
    _check(_lib.sq_smooth_quant_weight(_ptr(W, torch.bfloat16, "W", True), N, K, W.stride(0),
                                       _ptr(s, torch.float32, "s"), int(gran), _ptr(Wq, torch.int8, "Wq"),
                                       _ptr(w_scale, torch.float32, "w_scale"), wsp, wsb, _stream(stream)))
    return Wq, w_scale


def sq_smooth_quant_weight_noalloc(W, s, gran: int, Wq, w_scale, stream=None):
    """sq_smooth_quant_weight without a workspace (scratch lives in the library), for
    callers that cannot allocate device memory; calls overlapping on the GPU must not run
    concurrently."""
    torch = _torch()
    N, K = W.shape
    _check(_lib.sq_smooth_quant_weight_noalloc(_ptr(W, torch.bfloat16, "W", True), N, K, W.stride(0),
                                               _ptr(s, torch.float32, "s"), int(gran), _ptr(Wq, torch.int8, "Wq"),
                                               _ptr(w_scale, torch.float32, "w_scale"), _stream(stream)))
    return Wq, w_scale


def sq_quant_act_per_token(X, inv_s, Xq, x_scale, stream=None):
    torch = _torch()
    M, K = X.shape
    _check(_lib.sq_quant_act_per_token(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0),
                                       _ptr(inv_s, torch.float32, "inv_s"), _ptr(Xq, torch.int8, "Xq"),
                                       _ptr(x_scale, torch.float32, "x_scale"), _stream(stream)))
    return Xq, x_scale


def sq_int8_gemm_dequant(Xq, Wq, x_scale, w_scale, w_gran: int, bias, Y, acc_out=None, ws=None, stream=None):
    torch = _torch()
    M, K = Xq.shape
    N = Wq.shape[0]
    wsp, wsb = _ws(ws)
    _check(_lib.sq_int8_gemm_dequant(_ptr(Xq, torch.int8, "Xq"), _ptr(Wq, torch.int8, "Wq"),
                                     _ptr(x_scale, torch.float32, "x_scale"), _ptr(w_scale, torch.float32, "w_scale"),
                                     int(w_gran), _ptr(bias, torch.bfloat16, "bias"), _ptr(Y, torch.bfloat16, "Y"),
                                     M, N, K, _ptr(acc_out, torch.int32, "acc_out"), wsp, wsb, _stream(stream)))
    return Y


def llmint8_decomposed_linear(X, W, Wq, w_scale, threshold: float, bias, Y, mask_out=None, n_outliers_out=None,
                              acc_out=None, ws=None, stream=None):
    """mask_out is passed as a torch.int32 tensor of ceil(K/32) words (same bits as uint32)."""
    torch = _torch()
    M, K = X.shape
    N = W.shape[0]
    wsp, wsb = _ws(ws)
    _check(_lib.llmint8_decomposed_linear(
        _ptr(X, torch.bfloat16, "X"), _ptr(W, torch.bfloat16, "W"), _ptr(Wq, torch.int8, "Wq"),
        _ptr(w_scale, torch.float32, "w_scale"), float(threshold), _ptr(bias, torch.bfloat16, "bias"),
        _ptr(Y, torch.bfloat16, "Y"), M, N, K, _ptr(mask_out, torch.int32, "mask_out"),
        _ptr(n_outliers_out, torch.int32, "n_outliers_out"), _ptr(acc_out, torch.int32, "acc_out"), wsp, wsb,
        _stream(stream)))
    return Y


# ---------------------------------------------------------------- variants
def sq_quant_act_per_tensor(X, inv_s, Xq, x_scale, clip=None, ws=None, stream=None):
    """Per-tensor activation scale: dynamic (clip None, needs ws) or the calibrated *clip."""
    torch = _torch()
    M, K = X.shape
    wsp, wsb = _ws(ws)
    _check(_lib.sq_quant_act_per_tensor(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0),
                                        _ptr(inv_s, torch.float32, "inv_s"), _ptr(clip, torch.float32, "clip"),
                                        _ptr(Xq, torch.int8, "Xq"), _ptr(x_scale, torch.float32, "x_scale"), wsp, wsb,
                                        _stream(stream)))
    return Xq, x_scale


def sq_smooth_scale_ex(act_amax, W, alpha: float, normalize: bool, s, inv_s, stream=None):
    torch = _torch()
    N, K = W.shape
    _check(_lib.sq_smooth_scale_ex(_ptr(act_amax, torch.float32, "act_amax"), _ptr(W, torch.bfloat16, "W", True), N,
                                   K, W.stride(0), float(alpha), int(bool(normalize)), _ptr(s, torch.float32, "s"),
                                   _ptr(inv_s, torch.float32, "inv_s"), _stream(stream)))
    return s, inv_s


def sq_int8_gemm_dequant_ex(Xq, Wq, x_scale, x_gran: int, x_zero, w_scale, w_gran: int, w_rowsum, bias, Y,
                            acc_out=None, ws=None, stream=None):
    torch = _torch()
    M, K = Xq.shape
    N = Wq.shape[0]
    wsp, wsb = _ws(ws)
    _check(_lib.sq_int8_gemm_dequant_ex(
        _ptr(Xq, torch.int8, "Xq"), _ptr(Wq, torch.int8, "Wq"), _ptr(x_scale, torch.float32, "x_scale"), int(x_gran),
        _ptr(x_zero, torch.int32, "x_zero"), _ptr(w_scale, torch.float32, "w_scale"), int(w_gran),
        _ptr(w_rowsum, torch.int32, "w_rowsum"), _ptr(bias, torch.bfloat16, "bias"), _ptr(Y, torch.bfloat16, "Y"),
        M, N, K, _ptr(acc_out, torch.int32, "acc_out"), wsp, wsb, _stream(stream)))
    return Y


def sq_norm_smooth_quant(X, norm: int, gamma, beta, eps: float, inv_s, Xq, x_scale, mean_rstd=None, stream=None):
    torch = _torch()
    M, K = X.shape
    _check(_lib.sq_norm_smooth_quant(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0), int(norm),
                                     _ptr(gamma, torch.bfloat16, "gamma"), _ptr(beta, torch.bfloat16, "beta"),
                                     float(eps), _ptr(inv_s, torch.float32, "inv_s"), _ptr(Xq, torch.int8, "Xq"),
                                     _ptr(x_scale, torch.float32, "x_scale"),
                                     _ptr(mean_rstd, torch.float32, "mean_rstd"), _stream(stream)))
    return Xq, x_scale


def sq_act_mean_std_threshold(X, k: float, threshold, mean_std=None, ws=None, stream=None):
    torch = _torch()
    M, K = X.shape
    wsp, wsb = _ws(ws)
    _check(_lib.sq_act_mean_std_threshold(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0), float(k),
                                          _ptr(threshold, torch.float32, "threshold"),
                                          _ptr(mean_std, torch.float64, "mean_std"), wsp, wsb, _stream(stream)))
    return threshold


def llmint8_decomposed_linear_ex(X, W, Wq, w_scale, threshold, bias, Y, mask_out=None, n_outliers_out=None,
                                 acc_out=None, ws=None, stream=None):
    """llmint8_decomposed_linear with the threshold in a device fp32 [1] tensor."""
    torch = _torch()
    M, K = X.shape
    N = W.shape[0]
    wsp, wsb = _ws(ws)
    _check(_lib.llmint8_decomposed_linear_ex(
        _ptr(X, torch.bfloat16, "X"), _ptr(W, torch.bfloat16, "W"), _ptr(Wq, torch.int8, "Wq"),
        _ptr(w_scale, torch.float32, "w_scale"), _ptr(threshold, torch.float32, "threshold"),
        _ptr(bias, torch.bfloat16, "bias"), _ptr(Y, torch.bfloat16, "Y"), M, N, K,
        _ptr(mask_out, torch.int32, "mask_out"), _ptr(n_outliers_out, torch.int32, "n_outliers_out"),
        _ptr(acc_out, torch.int32, "acc_out"), wsp, wsb, _stream(stream)))
    return Y


def sq_act_abs_percentile(X, p: float, out, ws=None, stream=None):
    torch = _torch()
    M, K = X.shape
    wsp, wsb = _ws(ws)
    _check(_lib.sq_act_abs_percentile(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0), float(p),
                                      _ptr(out, torch.float32, "out"), wsp, wsb, _stream(stream)))
    return out


def sq_quant_act_per_token_asym(X, inv_s, Xq, x_scale, x_zero, stream=None):
    torch = _torch()
    M, K = X.shape
    _check(_lib.sq_quant_act_per_token_asym(_ptr(X, torch.bfloat16, "X", True), M, K, X.stride(0),
                                            _ptr(inv_s, torch.float32, "inv_s"), _ptr(Xq, torch.int8, "Xq"),
                                            _ptr(x_scale, torch.float32, "x_scale"),
                                            _ptr(x_zero, torch.int32, "x_zero"), _stream(stream)))
    return Xq, x_scale, x_zero


def sq_weight_row_sums(Wq, rowsum, stream=None):
    torch = _torch()
    N, K = Wq.shape
    _check(_lib.sq_weight_row_sums(_ptr(Wq, torch.int8, "Wq"), N, K, _ptr(rowsum, torch.int32, "rowsum"),
                                   _stream(stream)))
    return rowsum


# ---------------------------------------------------------------- 4-bit weights
# These calls run once per layer and token, so their checks are kept to a few microseconds.
_cuda_calls = None


def _cuda():
    """torch, and its calls for the current device and stream (the stream's handle, without making
    a Stream object for it, where torch has that), looked up once."""
    global _cuda_calls
    if _cuda_calls is None:
        torch = _torch()
        _cuda_calls = (torch, getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                       getattr(torch._C, "_cuda_getCurrentRawStream", None))
    return _cuda_calls


def _device(t, name):
    """Device index of a CUDA tensor, which must be the current device: the library launches there."""
    torch, current, _ = _cuda()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != current():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{current()}")
    return dev


def _on(stream, dev):
    """The handle of `stream`, or of the current one."""
    raw = _cuda()[2]
    return raw(dev) if stream is None and raw is not None else _stream(stream)


def _typed(t, dtype, name, dev):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{dev}")


def _dense(t, dtype, shape, name, dev):
    """Data pointer of a contiguous tensor of exactly this type and shape (None passes)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _typed(t, dtype, name, dev)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, dtype, name):
    """(data pointer, rows, columns, row stride) of a 2-D tensor with unit column stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    rows, columns = t.shape
    return t.data_ptr(), rows, columns, stride[0]


def sq_int4_weight_bytes(N: int, K: int) -> int:
    return int(_lib.sq_int4_weight_bytes(int(N), int(K)))


def _int4(torch, Wp, w_scale, w_zero, group, N, K, dev):
    groups = (-(-K // group) if group > 0 else 0, N)
    return (_dense(Wp, torch.uint8, (-(-N // 16) * -(-K // 128) * 1024,), "Wp", dev),
            _dense(w_scale, torch.bfloat16, groups, "w_scale", dev), _dense(w_zero, torch.uint8, groups, "w_zero", dev))


def sq_quant_weight_int4(W, s, group: int, Wp, w_scale, w_zero=None, stream=None):
    """4-bit codes and group scales of W [N, K] (times s); with w_zero, zero points too."""
    torch = _cuda()[0]
    dev = _device(W, "W")
    w, N, K, ldw = _rows(W, torch.bfloat16, "W")
    p, e, z = _int4(torch, Wp, w_scale, w_zero, group, N, K, dev)
    _check(_lib.sq_quant_weight_int4(w, N, K, ldw, _dense(s, torch.float32, (K,), "s", dev), group, p, e, z,
                                     _on(stream, dev)))
    return Wp, w_scale, w_zero


def sq_dequant_weight_int4(Wp, w_scale, w_zero, group: int, out, stream=None):
    """The bf16 values [N, K] (the shape of `out`) that a 4-bit weight stands for."""
    torch = _cuda()[0]
    dev = _device(out, "out")
    N, K = out.shape
    o = _dense(out, torch.bfloat16, (N, K), "out", dev)
    p, e, z = _int4(torch, Wp, w_scale, w_zero, group, N, K, dev)
    _check(_lib.sq_dequant_weight_int4(p, e, z, group, N, K, o, _on(stream, dev)))
    return out


def sq_int4_linear(X, Wp, w_scale, w_zero, group: int, bias, Y, stream=None):
    """Y [M, N] = X [M, K] times the 4-bit weight, plus bias; M <= 64."""
    torch = _cuda()[0]
    dev = _device(X, "X")
    x, M, K, ldx = _rows(X, torch.bfloat16, "X")
    N = Y.shape[-1]
    p, e, z = _int4(torch, Wp, w_scale, w_zero, group, N, K, dev)
    _check(_lib.sq_int4_linear(x, M, K, ldx, p, e, z, group, _dense(bias, torch.bfloat16, (N,), "bias", dev),
                               _dense(Y, torch.bfloat16, (M, N), "Y", dev), N, _on(stream, dev)))
    return Y


# ---------------------------------------------------------------- paged key-value cache
class _KvCacheStruct(C.Structure):
    _fields_ = [("type", C.c_int32), ("reserved", C.c_int32), ("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p),
                ("num_pages", _i64), ("heads", _i64), ("page_size", _i64), ("head_dim", _i64), ("page_stride", _i64),
                ("scale_page_stride", _i64)]


class KvCache:
    """Descriptor of a paged cache (sq_kv_cache) over the caller's tensors: k, v
    [num_pages, heads, page_size, head_dim] bf16, or int8 with fp32 scales k_scale, v_scale
    [num_pages, heads, page_size]; dense but for the page stride. Made once, passed to every
    call; it holds the tensors."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        torch = _torch()
        int8 = k.dtype == torch.int8
        if k.dim() != 4 or (not int8 and k.dtype != torch.bfloat16) or v.dtype != k.dtype:
            raise TypeError("k and v must be 4-D, both bfloat16 or both int8")
        if int8 != (k_scale is not None) or int8 != (v_scale is not None):
            raise ValueError("int8 caches have k_scale and v_scale, bf16 caches none")
        if int8 and (k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32):
            raise TypeError("cache scales must be float32")
        pages, heads, page_size, dim = k.shape
        for t, shape, dense in ((k, k.shape, (page_size * dim, dim, 1)), (v, k.shape, (page_size * dim, dim, 1)),
                                (k_scale, k.shape[:3], (page_size, 1)), (v_scale, k.shape[:3], (page_size, 1))):
            if t is not None and (t.shape != shape or any(s != d for s, d, n in zip(t.stride()[1:], dense, shape[1:])
                                                          if n > 1)):
                raise ValueError("cache tensors must have one shape and be dense within a page")
        if not k.is_cuda or any(t is not None and t.device != k.device for t in (v, k_scale, v_scale)):
            raise ValueError("cache tensors must be on one CUDA device")

        def stride(a, b):
            if pages == 1:
                return a.numel()
            if a.stride(0) != b.stride(0):
                raise ValueError("k and v (and their scales) must share one page stride")
            return a.stride(0)

        self.tensors = (k, v, k_scale, v_scale)
        self.device = k.get_device()
        self.heads, self.head_dim = heads, dim
        self.struct = _KvCacheStruct(
            SQ_KV_INT8 if int8 else SQ_KV_BF16, 0, k.data_ptr(), v.data_ptr(),
            k_scale.data_ptr() if int8 else None, v_scale.data_ptr() if int8 else None, pages, heads, page_size, dim,
            stride(k, v), stride(k_scale, v_scale) if int8 else 0)
        self.ref = C.addressof(self.struct)


def _heads(t, bf16, heads, dim, name, dev):
    """(data pointer, token stride) of a bf16 [tokens, heads, dim] tensor dense within a token."""
    if t.dtype is not bf16 or t.get_device() != dev:
        _typed(t, bf16, name, dev)
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or stride[2] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}], dense within a token")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * dim


def sq_rope_kv_append(q, k, v, cos, sin, positions, slots, cache: KvCache, q_out, interleaved: bool = False,
                      stream=None):
    """Rotate q and k by position, write q_out, append k and v to the cache's slots. q and q_out
    may be None; cos, sin [max_pos, rot_dim / 2] and positions may be None (no rotation)."""
    torch = _cuda()[0]
    dev = _device(k, "k")
    if dev != cache.device:
        raise ValueError(f"cache on cuda:{cache.device}, k on cuda:{dev}")
    heads, D = cache.heads, cache.head_dim
    kp, ldk = _heads(k, torch.bfloat16, heads, D, "k", dev)
    vp, ldv = _heads(v, torch.bfloat16, heads, D, "v", dev)
    T = k.shape[0]
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out must be given together")
    if (cos is None) != (sin is None) or (cos is None) != (positions is None):
        raise ValueError("cos, sin and positions must be given together")
    H, qp, ldq, op = 0, None, 0, None
    if q is not None:
        H = q.shape[1]
        qp, ldq = _heads(q, torch.bfloat16, H, D, "q", dev)
        op = _dense(q_out, torch.bfloat16, (T, H, D), "q_out", dev)
    if v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("q, k and v must have the same number of tokens")
    max_pos, half, cp, sp, pp = 0, 0, None, None, None
    if cos is not None:
        max_pos, half = cos.shape
        cp = _dense(cos, torch.float32, (max_pos, half), "cos", dev)
        sp = _dense(sin, torch.float32, (max_pos, half), "sin", dev)
        pp = _dense(positions, torch.int32, (T,), "positions", dev)
    _check(_lib.sq_rope_kv_append(qp, ldq, kp, ldk, vp, ldv, T, H, cp, sp, max_pos, 2 * half,
                                  1 if interleaved else 0, pp,
                                  _dense(slots, torch.int32, (T,), "slots", dev), cache.ref, op, _on(stream, dev)))
    return q_out


def sq_paged_attention(q, cache: KvCache, block_table, seq_lens, scale: float, out, lse=None, window: int = 0, ws=None,
                       stream=None):
    """out [B, H, D]: attention of one token per sequence over the cache; lse [B, H] fp32 too."""
    torch = _cuda()[0]
    dev = _device(q, "q")
    if dev != cache.device:
        raise ValueError(f"cache on cuda:{cache.device}, q on cuda:{dev}")
    if q.dim() != 3:
        raise ValueError("q must be [sequences, heads, head_dim]")
    B, H, D = q.shape
    qp, ldq = _heads(q, torch.bfloat16, H, cache.head_dim, "q", dev)
    _typed(block_table, torch.int32, "block_table", dev)
    shape, stride = block_table.shape, block_table.stride()
    if len(shape) != 2 or shape[0] != B or (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"block_table must be [{B}, max_pages] with unit column stride")
    wsp, wsb = None, 0
    if ws is not None:
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be a contiguous tensor on cuda:{dev}")
        wsp, wsb = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(_lib.sq_paged_attention(
        qp, ldq, B, H, cache.ref, block_table.data_ptr(), stride[0] if B > 1 else shape[1], shape[1],
        _dense(seq_lens, torch.int32, (B,), "seq_lens", dev), window, scale,
        _dense(out, torch.bfloat16, (B, H, D), "out", dev), _dense(lse, torch.float32, (B, H), "lse", dev), wsp, wsb,
        _on(stream, dev)))
    return out


def sq_workspace_size(op: int, M: int, N: int, K: int) -> int:
    return int(_lib.sq_workspace_size(int(op), int(M), int(N), int(K)))


def sq_sync_status(stream=None):
    _check(_lib.sq_sync_status(_stream(stream)))


def sq_kernel_launch_count() -> int:
    return int(_lib.sq_kernel_launch_count())


def sq_debug_guard_margin(margin: int):
    _check(_lib.sq_debug_guard_margin(int(margin)))


def sq_debug_arm_fault(fault: int, wait_limit_ns: int = 0):
    _lib.sq_debug_arm_fault(int(fault), int(wait_limit_ns))


GEMM_PLAN_FIELDS = ("path", "swap", "bn", "whole_tiles", "split_tiles", "splits", "kb_per_split")
GEMM_PATH_CUDA_CORES, GEMM_PATH_TENSOR, GEMM_PATH_TENSOR_PAIRS = 0, 1, 2


def sq_debug_gemm_plan(M: int, N: int, K: int, outliers: bool = False) -> dict:
    """The launch plan of the GEMM for an M x N x K product (host only, no device)."""
    out = (C.c_int64 * 7)()
    _check(_lib.sq_debug_gemm_plan(int(M), int(N), int(K), 1 if outliers else 0, C.cast(out, C.c_void_p)))
    return dict(zip(GEMM_PLAN_FIELDS, (int(v) for v in out)))


def workspace(op: int, M: int, N: int, K: int, device="cuda"):
    """A uint8 torch tensor of sq_workspace_size(op, M, N, K) bytes (None if 0), zero-filled."""
    torch = _torch()
    n = sq_workspace_size(op, M, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None
