"""Python binding of the Spense C interface (``include/spense.h``).

Argument marshalling only: every step of the layer runs in the HIP library
``libspense.so`` built next to this file.  There is no Python or CPU fallback;
if the library is missing every call raises.

Tensors are passed by device pointer (``tensor.data_ptr()``); torch is used
only to own device memory and to name the current HIP stream.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import numpy as np

DT_F32 = 0
DT_BF16 = 1
DT_FP8 = 2
DT_MX4 = 3

SPENSE_OK = 0
SPENSE_EINVAL = -1
SPENSE_EUNSUPPORTED = -2
SPENSE_ENOMEM = -3
SPENSE_EHIP = -4
SPENSE_ESCRATCH = -5

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspense.so")

_lib_handle = None


class SpenseError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib()
        msg = lib.spense_strerror(status).decode()
        if status == SPENSE_EHIP:
            msg += f" (hipError_t {lib.spense_last_hip_error()})"
        super().__init__(f"{where}: {msg} [{status}]")
        self.status = status


class LayerInfo(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("K_s", ctypes.c_int64), ("K_d", ctypes.c_int64),
        ("wdtype", ctypes.c_int32), ("gather", ctypes.c_int32),
        ("weight_bytes", ctypes.c_int64), ("device_bytes", ctypes.c_int64),
        ("split", ctypes.c_int32), ("N_s", ctypes.c_int64), ("N_d", ctypes.c_int64),
    ]


def _lib():
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m sparse_dense_gemm_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
    lib.spense_pack.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, f64, vp, ctypes.POINTER(vp)]
    lib.spense_pack.restype = ctypes.c_int
    lib.spense_pack_rows.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, f64, vp, ctypes.POINTER(vp)]
    lib.spense_pack_rows.restype = ctypes.c_int
    lib.spense_export_rows.argtypes = [vp, vp, vp, vp, vp, vp, vp]
    lib.spense_export_rows.restype = ctypes.c_int
    lib.spense_pack_glu.argtypes = [vp, vp, i32, i64, i64, i64, i64, vp, vp, vp, i64, f64, vp, ctypes.POINTER(vp)]
    lib.spense_pack_glu.restype = ctypes.c_int
    lib.spense_glu.argtypes = [vp, vp, i64, i64, vp, i64, vp, i32, i64, vp]
    lib.spense_glu.restype = ctypes.c_int
    lib.spense_score_glu.argtypes = [vp, vp, i32, i64, i64, i64, i64, vp, vp, vp, i64, i64, vp, i64, vp, vp]
    lib.spense_score_glu.restype = ctypes.c_int
    lib.spense_select_dense.argtypes = [vp, i64, i64, vp, vp]
    lib.spense_select_dense.restype = ctypes.c_int
    lib.spense_linear.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.spense_linear.restype = ctypes.c_int
    lib.spense_linear_splits.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, i32, vp]
    lib.spense_linear_noalloc.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.spense_linear_noalloc.restype = ctypes.c_int
    lib.spense_quantize_tokens.restype = ctypes.c_int
    lib.spense_quantize_tokens.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp]
    lib.spense_linear_w8a8.restype = ctypes.c_int
    lib.spense_linear_w8a8.argtypes = [vp, vp, i64, i64, vp, i32, i64, i32, vp]
    lib.spense_linear_splits.restype = ctypes.c_int
    lib.spense_quantize_mx4.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp]
    lib.spense_quantize_mx4.restype = ctypes.c_int
    lib.spense_dequantize_mx4.argtypes = [vp, i64, vp, i64, i64, i64, vp, i32, i64, vp]
    lib.spense_dequantize_mx4.restype = ctypes.c_int
    lib.spense_pack_mx4.argtypes = [vp, i64, vp, i64, i64, i64, vp, ctypes.POINTER(vp)]
    lib.spense_pack_mx4.restype = ctypes.c_int
    lib.spense_linear_w4a4.argtypes = [vp, vp, i64, i64, vp, i32, i64, vp]
    lib.spense_linear_w4a4.restype = ctypes.c_int
    lib.spense_pack_experts.argtypes = [vp, i32, vp, i64, i64, i64, i64, i64, i32, vp, ctypes.POINTER(vp)]
    lib.spense_pack_experts.restype = ctypes.c_int
    lib.spense_experts_linear.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.spense_experts_linear.restype = ctypes.c_int
    lib.spense_route_workspace.argtypes = [i64, i64, i32]
    lib.spense_route_workspace.restype = i64
    lib.spense_route.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.spense_route.restype = ctypes.c_int
    lib.spense_experts_combine.argtypes = [vp, i32, i64, i64, vp, vp, i64, i32, i64, vp, i32, i64, vp]
    lib.spense_experts_combine.restype = ctypes.c_int
    lib.spense_info.argtypes = [vp, ctypes.POINTER(LayerInfo)]
    lib.spense_info.restype = ctypes.c_int
    lib.spense_export.argtypes = [vp, vp, vp, vp, vp, vp, vp]
    lib.spense_export.restype = ctypes.c_int
    lib.spense_free.argtypes = [vp]
    lib.spense_free.restype = ctypes.c_int
    lib.spense_strerror.argtypes = [ctypes.c_int]
    lib.spense_strerror.restype = ctypes.c_char_p
    lib.spense_last_hip_error.argtypes = []
    lib.spense_last_hip_error.restype = ctypes.c_int
    lib.spense_abi_version.argtypes = []
    lib.spense_abi_version.restype = ctypes.c_int
    _lib_handle = lib
    return lib


def _check(status: int, where: str):
    if status != SPENSE_OK:
        raise SpenseError(status, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        torch = _torch()
        if _raw_stream is not None:  # the handle itself, without a Stream object around it (0.1 instead of 2.7 us)
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_torch_module = None
_raw_stream = None
_dtypes = {}


def _torch():
    global _torch_module, _raw_stream, _dtypes
    if _torch_module is None:
        import torch

        # each name is bound once it is whole, the module last: another thread may look at any of them meanwhile
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _dtypes = {torch.float32: DT_F32, torch.bfloat16: DT_BF16, torch.float8_e4m3fn: DT_FP8, torch.uint8: DT_FP8}
        _torch_module = torch
    return _torch_module


def dtype_of(t) -> int:
    if not _dtypes:
        _torch()
    d = _dtypes.get(t.dtype)
    if d is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return d


def _need_dtype(t, dtype, what: str) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{what} is {dtype}, not {t.dtype}")


def _matrix(t, what: str):
    """Rows, columns and row stride of a matrix that is contiguous along a row."""
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what} {rows} x {cols} is not contiguous along a row")
    return rows, cols, ld


def _too_small(what: str, rows: int, cols: int):
    raise ValueError(f"{what} does not hold {rows} rows of {cols} columns")


def _need_flat(t, dtype, n: int, what: str) -> None:
    """t is contiguous, of this type, and holds at least n values."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} is {dtype}, not {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what} {tuple(t.shape)} does not hold {n} contiguous values")


def spense_pack(W, wdtype: Optional[int] = None, *, scales=None, dense_cols=None, dense_fraction: float = 0.0,
                N: Optional[int] = None, K: Optional[int] = None, ldw: Optional[int] = None, stream=None) -> int:
    """Pack a weight matrix; returns the opaque handle (an int)."""
    if wdtype is None:
        wdtype = dtype_of(W)
    if N is None:
        N = W.shape[0]
    if K is None:
        K = W.shape[1]
    if ldw is None:
        ldw = W.stride(0) if hasattr(W, "stride") else K
    cols_ptr = None
    n_dense = 0
    if dense_cols is not None:
        cols = np.ascontiguousarray(np.asarray(dense_cols, dtype=np.int32).ravel())
        n_dense = cols.size
        # an explicit empty set still needs a non-null pointer
        buf = cols if n_dense else np.zeros(1, dtype=np.int32)
        cols_ptr = buf.ctypes.data
    h = ctypes.c_void_p()
    st = _lib().spense_pack(_ptr(W), wdtype, N, K, ldw, _ptr(scales), cols_ptr, n_dense, float(dense_fraction),
                            _stream(stream), ctypes.byref(h))
    _check(st, "spense_pack")
    return h.value


def spense_pack_rows(W, wdtype: Optional[int] = None, *, scales=None, dense_rows=None, dense_fraction: float = 0.0,
                     N: Optional[int] = None, K: Optional[int] = None, ldw: Optional[int] = None,
                     stream=None) -> int:
    """Pack an output-split layer (dense rows | 2:4 rows); returns the opaque handle (an int)."""
    if wdtype is None:
        wdtype = dtype_of(W)
    if N is None:
        N = W.shape[0]
    if K is None:
        K = W.shape[1]
    if ldw is None:
        ldw = W.stride(0) if hasattr(W, "stride") else K
    rows_ptr = None
    n_dense = 0
    if dense_rows is not None:
        rows = np.ascontiguousarray(np.asarray(dense_rows, dtype=np.int32).ravel())
        n_dense = rows.size
        buf = rows if n_dense else np.zeros(1, dtype=np.int32)
        rows_ptr = buf.ctypes.data
    h = ctypes.c_void_p()
    st = _lib().spense_pack_rows(_ptr(W), wdtype, N, K, ldw, _ptr(scales), rows_ptr, n_dense, float(dense_fraction),
                                 _stream(stream), ctypes.byref(h))
    _check(st, "spense_pack_rows")
    return h.value


def spense_export_rows(h: int, vals=None, meta=None, mask=None, dense=None, stream=None) -> np.ndarray:
    """Write an output-split layer's canonical form into the given device tensors; returns rho (numpy int32)."""
    info = spense_info(h)
    rho = np.empty(info["N"], dtype=np.int32)
    st = _lib().spense_export_rows(h, _ptr(vals), _ptr(meta), _ptr(mask), _ptr(dense), rho.ctypes.data,
                                   _stream(stream))
    _check(st, "spense_export_rows")
    return rho


def spense_pack_glu(W_gu, W_down, wdtype: int, *, H: int, I: int, s_gu=None, s_down=None, dense_idx=None,
                    dense_fraction: float = 0.0, stream=None) -> int:
    """Pack a GLU block: W_gu = [gate; up] as [2I, H], W_down [H, I]; returns the handle."""
    idx_ptr, n_dense = None, 0
    if dense_idx is not None:
        idx = np.ascontiguousarray(np.asarray(dense_idx, dtype=np.int32).ravel())
        n_dense = idx.size
        buf = idx if n_dense else np.zeros(1, dtype=np.int32)
        idx_ptr = buf.ctypes.data
    ld_gu = W_gu.stride(0) if hasattr(W_gu, "stride") else H
    ld_down = W_down.stride(0) if hasattr(W_down, "stride") else I
    h = ctypes.c_void_p()
    st = _lib().spense_pack_glu(_ptr(W_gu), _ptr(W_down), wdtype, H, I, ld_gu, ld_down, _ptr(s_gu), _ptr(s_down),
                                idx_ptr, n_dense, float(dense_fraction), _stream(stream), ctypes.byref(h))
    _check(st, "spense_pack_glu")
    return h.value


def spense_glu(h: int, X, A, Y, *, M: Optional[int] = None, stream=None) -> None:
    """GLU block forward: A (bf16 [M, >= I]) receives silu(gate) * up in rho order, Y the block output."""
    M = X.shape[0] if M is None else M
    ydtype = dtype_of(Y)
    st = _lib().spense_glu(h, _ptr(X), M, X.stride(0), _ptr(A), A.stride(0), _ptr(Y), ydtype, Y.stride(0),
                           _stream(stream))
    _check(st, "spense_glu")


def spense_score_glu(W_gu, W_down, wdtype: int, *, H: int, I: int, X_cal, A_cal, score, s_gu=None, s_down=None,
                     stream=None) -> None:
    """SpenseGPT+ scores of the intermediate indices of a GLU block into `score` (float32 [I], device)."""
    ld_gu = W_gu.stride(0) if hasattr(W_gu, "stride") else H
    ld_down = W_down.stride(0) if hasattr(W_down, "stride") else I
    st = _lib().spense_score_glu(_ptr(W_gu), _ptr(W_down), wdtype, H, I, ld_gu, ld_down, _ptr(s_gu), _ptr(s_down),
                                 _ptr(X_cal), X_cal.shape[0], X_cal.stride(0), _ptr(A_cal), A_cal.stride(0),
                                 _ptr(score), _stream(stream))
    _check(st, "spense_score_glu")


def spense_select_dense(score, k: int, stream=None) -> np.ndarray:
    """Indices of the k highest scores (ties to the lower index), ascending, as numpy int32."""
    out = np.zeros(max(k, 1), dtype=np.int32)
    st = _lib().spense_select_dense(_ptr(score), score.numel(), k, out.ctypes.data, _stream(stream))
    _check(st, "spense_select_dense")
    return out[:k]


def spense_linear(h: int, X, Y, *, xdtype: Optional[int] = None, ydtype: Optional[int] = None,
                  M: Optional[int] = None, ldx: Optional[int] = None, ldy: Optional[int] = None, stream=None) -> None:
    """Y = X . W^T through the packed layer (asynchronous on the stream)."""
    spense_linear_splits(h, X, Y, 0, xdtype=xdtype, ydtype=ydtype, M=M, ldx=ldx, ldy=ldy, stream=stream)


def spense_linear_splits(h: int, X, Y, splits: int, *, xdtype: Optional[int] = None, ydtype: Optional[int] = None,
                         M: Optional[int] = None, ldx: Optional[int] = None, ldy: Optional[int] = None,
                         stream=None) -> None:
    if xdtype is None:
        xdtype = dtype_of(X)
    if ydtype is None:
        ydtype = dtype_of(Y)
    if M is None:
        M = X.shape[0]
    if ldx is None:
        ldx = X.stride(0)
    if ldy is None:
        ldy = Y.stride(0)
    st = _lib().spense_linear_splits(h, _ptr(X), xdtype, M, ldx, _ptr(Y), ydtype, ldy, splits, _stream(stream))
    _check(st, "spense_linear")


def spense_linear_noalloc(h: int, X, Y, *, xdtype: Optional[int] = None, ydtype: Optional[int] = None,
                          M: Optional[int] = None, ldx: Optional[int] = None, ldy: Optional[int] = None,
                          stream=None) -> None:
    """spense_linear with its workspaces in the library's fixed device scratch (allocates nothing)."""
    xdtype = dtype_of(X) if xdtype is None else xdtype
    ydtype = dtype_of(Y) if ydtype is None else ydtype
    M = X.shape[0] if M is None else M
    ldx = X.stride(0) if ldx is None else ldx
    ldy = Y.stride(0) if ldy is None else ldy
    st = _lib().spense_linear_noalloc(h, _ptr(X), xdtype, M, ldx, _ptr(Y), ydtype, ldy, _stream(stream))
    _check(st, "spense_linear_noalloc")


def spense_quantize_tokens(X, Xq, sx, *, M: Optional[int] = None, K: Optional[int] = None,
                           ldx: Optional[int] = None, ldq: Optional[int] = None, stream=None) -> None:
    """Per-token e4m3 codes of bf16 X into Xq (uint8 [M, K]) and the token scales into sx (float32 [M])."""
    if M is None:
        M = X.shape[0]
    if K is None:
        K = X.shape[1]
    if ldx is None:
        ldx = X.stride(0)
    if ldq is None:
        ldq = Xq.stride(0)
    st = _lib().spense_quantize_tokens(_ptr(X), M, K, ldx, _ptr(Xq), ldq, _ptr(sx), _stream(stream))
    _check(st, "spense_quantize_tokens")


def spense_linear_w8a8(h: int, X, Y, *, splits: int = 0, ydtype: Optional[int] = None, M: Optional[int] = None,
                       ldx: Optional[int] = None, ldy: Optional[int] = None, stream=None) -> None:
    """Y = (per-token e4m3 X) . W^T on an e4m3 input-split layer, X bfloat16 (asynchronous on the stream)."""
    _need_dtype(X, _torch().bfloat16, "X")
    if ydtype is None:
        ydtype = dtype_of(Y)
    if M is None:
        M = X.shape[0]
    if ldx is None:
        ldx = X.stride(0)
    if ldy is None:
        ldy = Y.stride(0)
    st = _lib().spense_linear_w8a8(h, _ptr(X), M, ldx, _ptr(Y), ydtype, ldy, splits, _stream(stream))
    _check(st, "spense_linear_w8a8")


def spense_quantize_mx4(X, codes, scales, *, xdtype: Optional[int] = None, stream=None) -> None:
    """mx4 form of X [M, K]: codes (uint8 [M, >= (K+1)/2]) and exponent bytes (uint8 [M, >= ceil(K/32)])."""
    if xdtype is None:
        xdtype = dtype_of(X)
    else:
        _need_width(X, xdtype, "X")
    M, K, ldx = _matrix(X, "X")
    ldc, lds = _mx4_strides(codes, scales, M, K)
    st = _lib().spense_quantize_mx4(X.data_ptr(), xdtype, M, K, ldx, codes.data_ptr(), ldc, scales.data_ptr(), lds,
                                    _stream(stream))
    _check(st, "spense_quantize_mx4")


def spense_dequantize_mx4(codes, scales, Y, *, ydtype: Optional[int] = None, stream=None) -> None:
    """The numbers an mx4 matrix stands for, into Y [M, K] (float32 or bfloat16)."""
    if ydtype is None:
        ydtype = dtype_of(Y)
    else:
        _need_width(Y, ydtype, "Y")
    M, K, ldy = _matrix(Y, "Y")
    ldc, lds = _mx4_strides(codes, scales, M, K)
    st = _lib().spense_dequantize_mx4(codes.data_ptr(), ldc, scales.data_ptr(), lds, M, K, Y.data_ptr(), ydtype, ldy,
                                      _stream(stream))
    _check(st, "spense_dequantize_mx4")


_WIDTH = {DT_F32: 4, DT_BF16: 2, DT_FP8: 1, DT_MX4: 1}


def _need_width(t, dtype: int, what: str) -> None:
    """A type named by the caller has the width of t's elements (types the library refuses are left to it)."""
    if t.element_size() != _WIDTH.get(dtype, t.element_size()):
        raise TypeError(f"{what} of {t.dtype} does not hold elements of type {dtype}")


def _mx4_strides(codes, scales, rows: int, K: int):
    """Row strides of an mx4 matrix of at least rows x K."""
    crows, cbytes, ldc = _matrix(codes, "codes")
    srows, sbytes, lds = _matrix(scales, "scales")
    if crows < rows or srows < rows or cbytes < (K + 1) // 2 or sbytes < (K + 31) // 32:
        raise ValueError(f"codes {crows} x {cbytes} and scales {srows} x {sbytes} do not hold {rows} x {K} mx4")
    if codes.element_size() != 1 or scales.element_size() != 1:
        raise ValueError("codes and scales are bytes")
    return ldc, lds


def spense_pack_mx4(codes, scales, *, N: Optional[int] = None, K: Optional[int] = None, stream=None) -> int:
    """Pack an mx4 weight matrix [N, K] (K: twice the code bytes of a row unless given); returns the handle."""
    N = codes.shape[0] if N is None else N
    K = 2 * codes.shape[1] if K is None else K
    ldc, lds = _mx4_strides(codes, scales, N, K)
    h = ctypes.c_void_p()
    st = _lib().spense_pack_mx4(codes.data_ptr(), ldc, scales.data_ptr(), lds, N, K, _stream(stream), ctypes.byref(h))
    _check(st, "spense_pack_mx4")
    return h.value


class _Dims(NamedTuple):
    """What the calls on an mx4 layer or on experts' layers check tensors against."""
    K: int
    columns: int  # of an output row
    experts: int


def _dims(h: int) -> Optional[_Dims]:
    """None for a handle of another kind, which the library refuses."""
    info = LayerInfo()
    _check(_lib().spense_info(h, ctypes.byref(info)), "spense_info")
    return _Dims(info.K, info.N_d, info.N_s) if info.split in (3, 4) else None


def spense_linear_w4a4(h: int, X, Y, *, M: Optional[int] = None, stream=None) -> None:
    """Y = mx4(X) . W^T on an mx4 layer, X bfloat16 (asynchronous on the stream)."""
    _linear_w4a4(h, _dims(h), X, Y, M, stream)


def _linear_w4a4(h, dims, X, Y, M, stream):
    _need_dtype(X, _torch().bfloat16, "X")
    xrows, xcols, ldx = _matrix(X, "X")
    yrows, ycols, ldy = _matrix(Y, "Y")
    M = xrows if M is None else M
    if dims:
        if xrows < M or xcols < dims.K:
            _too_small("X", M, dims.K)
        if yrows < M or ycols < dims.columns:
            _too_small("Y", M, dims.columns)
    st = _lib().spense_linear_w4a4(h, X.data_ptr(), M, ldx, Y.data_ptr(), dtype_of(Y), ldy, _stream(stream))
    _check(st, "spense_linear_w4a4")


def spense_pack_experts(W, wdtype: Optional[int] = None, *, scales=None, K: Optional[int] = None, glu: bool = False,
                        stream=None) -> int:
    """Pack experts' weights: W bf16 [E, N, K], or mx4 codes [E, N, bytes] with exponent bytes [E, N, ceil(K/32)]."""
    wdtype = dtype_of(W) if wdtype is None else wdtype
    E, N = W.shape[0], W.shape[1]
    if K is None:
        K = 2 * W.shape[2] if wdtype == DT_MX4 else W.shape[2]
    W2 = _rows_in_line(W)
    _need_width(W, wdtype, "W")
    if wdtype == DT_BF16 and W.shape[2] < K:
        _too_small("W", E * N, K)
    s2 = None if scales is None else _rows_in_line(scales)
    if wdtype == DT_MX4 and s2 is not None:
        _mx4_strides(W2, s2, E * N, K)
    h = ctypes.c_void_p()
    st = _lib().spense_pack_experts(W2.data_ptr(), wdtype, _ptr(s2), E, N, K, W2.stride(0),
                                    0 if s2 is None else s2.stride(0), int(glu), _stream(stream), ctypes.byref(h))
    _check(st, "spense_pack_experts")
    return h.value


def _rows_in_line(t):
    """[E, N, C] as [E * N, C] without a copy."""
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[0] > 1 and t.stride(0) != t.shape[1] * t.stride(1)):
        raise ValueError("experts' matrices are [E, N, columns], one after the other, contiguous along a row")
    return t.as_strided((t.shape[0] * t.shape[1], t.shape[2]), (t.stride(1), 1))


def spense_experts_linear(h: int, X, offsets, Y, *, rows=None, adtype: int = DT_BF16, R: Optional[int] = None,
                          stream=None) -> None:
    """Rows of X (bfloat16) grouped by expert (offsets int32 [E + 1], rows int32 [R] if X is not grouped itself)
    into Y [R, ...]."""
    _experts_linear(h, _dims(h), X, offsets, Y, rows, adtype, R, stream)


def _experts_linear(h, dims, X, offsets, Y, rows, adtype, R, stream):
    torch = _torch()
    i32 = torch.int32
    if X.dtype is not torch.bfloat16:
        _need_dtype(X, torch.bfloat16, "X")
    M, xcols, ldx = _matrix(X, "X")
    yrows, ycols, ldy = _matrix(Y, "Y")
    if R is None:
        R = yrows
    if dims:
        K, columns, experts = dims
        if xcols < K:
            _too_small("X", M, K)
        if yrows < R or ycols < columns:
            _too_small("Y", R, columns)
        if offsets.dtype is not i32 or offsets.numel() <= experts or not offsets.is_contiguous():
            _need_flat(offsets, i32, experts + 1, "offsets")
    if rows is not None and (rows.dtype is not i32 or rows.numel() < R or not rows.is_contiguous()):
        _need_flat(rows, i32, R, "rows")
    st = _lib().spense_experts_linear(h, X.data_ptr(), adtype, M, ldx, None if rows is None else rows.data_ptr(),
                                      offsets.data_ptr(), R, Y.data_ptr(), dtype_of(Y), ldy, _stream(stream))
    _check(st, "spense_experts_linear")


@functools.lru_cache(maxsize=256)
def spense_route_workspace(T: int, E: int, k: int) -> int:
    """Bytes of workspace spense_route needs."""
    n = _lib().spense_route_workspace(T, E, k)
    if n < 0:
        _check(int(n), "spense_route_workspace")
    return n


def spense_route(logits, k: int, ids, weights, offsets, rows, pos, work=None, *, renormalize: bool = True,
                 stream=None) -> None:
    """Experts of every token (ids int32, weights float32 [T, k]) and the tokens grouped by expert
    (offsets int32 [E + 1], rows int32 [T * k], pos int32 [T, k])."""
    T, E, ldl = _matrix(logits, "logits")
    n = T * k
    if ids.numel() < n or weights.numel() < n or rows.numel() < n or pos.numel() < n or offsets.numel() < E + 1:
        raise ValueError("ids, weights, rows and pos hold T * k values, offsets E + 1")
    need = spense_route_workspace(T, E, k)
    if need and (work is None or work.numel() * work.element_size() < need or not work.is_contiguous()):
        raise ValueError(f"spense_route needs {need} contiguous bytes of workspace")
    torch = _torch()
    i32 = torch.int32
    if not (ids.dtype is i32 and pos.dtype is i32 and rows.dtype is i32 and offsets.dtype is i32
            and weights.dtype is torch.float32 and ids.is_contiguous() and pos.is_contiguous()
            and rows.is_contiguous() and offsets.is_contiguous() and weights.is_contiguous()):
        for t, what in ((ids, "ids"), (pos, "pos"), (rows, "rows"), (offsets, "offsets")):
            _need_flat(t, i32, 0, what)
        _need_flat(weights, torch.float32, 0, "weights")
    st = _lib().spense_route(logits.data_ptr(), dtype_of(logits), T, E, ldl, k, int(renormalize),
                             ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(),
                             None if work is None else work.data_ptr(), _stream(stream))
    _check(st, "spense_route")


def spense_experts_combine(O, pos, weights, Y, *, stream=None) -> None:
    """Y[t] = sum_j weights[t, j] O[pos[t, j]] (pos int32, weights float32 [T, k])."""
    torch = _torch()
    T, k = pos.shape
    R, ocols, ldo = _matrix(O, "O")
    yrows, N, ldy = _matrix(Y, "Y")
    if ocols < N:
        _too_small("O", R, N)
    if yrows < T:
        _too_small("Y", T, N)
    _need_flat(pos, torch.int32, 0, "pos")
    _need_flat(weights, torch.float32, T * k, "weights")
    st = _lib().spense_experts_combine(O.data_ptr(), dtype_of(O), R, ldo, pos.data_ptr(), weights.data_ptr(), T, k, N,
                                       Y.data_ptr(), dtype_of(Y), ldy, _stream(stream))
    _check(st, "spense_experts_combine")


def spense_info(h: int) -> dict:
    info = LayerInfo()
    _check(_lib().spense_info(h, ctypes.byref(info)), "spense_info")
    return {f: getattr(info, f) for f, _ in LayerInfo._fields_}


def spense_export(h: int, vals=None, meta=None, mask=None, dense=None, stream=None) -> np.ndarray:
    """Write the canonical packed form into the given device tensors; returns pi (numpy int32)."""
    info = spense_info(h)
    pi = np.empty(info["K"], dtype=np.int32)
    st = _lib().spense_export(h, _ptr(vals), _ptr(meta), _ptr(mask), _ptr(dense), pi.ctypes.data, _stream(stream))
    _check(st, "spense_export")
    return pi


def spense_free(h: int) -> None:
    _check(_lib().spense_free(h), "spense_free")


def spense_abi_version() -> int:
    return _lib().spense_abi_version()


class _Owned:
    """Owns a packed layer's handle."""

    handle = None

    def close(self):
        if self.handle:
            spense_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SpenseLinear(_Owned):
    """Owns one packed layer; ``layer(X, Y)`` runs spense_linear."""

    def __init__(self, W, wdtype: Optional[int] = None, **kw):
        self.handle = spense_pack(W, wdtype, **kw)
        self.info = spense_info(self.handle)

    def __call__(self, X, Y, splits: int = 0, stream=None):
        spense_linear_splits(self.handle, X, Y, splits, stream=stream)
        return Y


class SpenseLinearMx4(_Owned):
    """Owns one packed mx4 layer; ``layer(X, Y)`` runs spense_linear, ``layer.w4a4(X, Y)`` spense_linear_w4a4."""

    def __init__(self, codes, scales, **kw):
        self.handle = spense_pack_mx4(codes, scales, **kw)
        self.info = spense_info(self.handle)
        self._dims = _dims(self.handle)

    def __call__(self, X, Y, stream=None):
        M, xcols, ldx = _matrix(X, "X")
        yrows, ycols, ldy = _matrix(Y, "Y")
        if xcols < self._dims.K:
            _too_small("X", M, self._dims.K)
        if yrows < M or ycols < self._dims.columns:
            _too_small("Y", M, self._dims.columns)
        spense_linear(self.handle, X, Y, M=M, ldx=ldx, ldy=ldy, stream=stream)
        return Y

    def w4a4(self, X, Y, stream=None):
        _linear_w4a4(self.handle, self._dims, X, Y, None, stream)
        return Y


class SpenseExperts(_Owned):
    """Owns the packed layers of a set of experts; ``experts(X, offsets, Y, rows=...)`` runs spense_experts_linear."""

    def __init__(self, W, wdtype: Optional[int] = None, **kw):
        self.handle = spense_pack_experts(W, wdtype, **kw)
        self.info = spense_info(self.handle)
        self._dims = _dims(self.handle)

    def __call__(self, X, offsets, Y, *, rows=None, adtype: int = DT_BF16, stream=None):
        _experts_linear(self.handle, self._dims, X, offsets, Y, rows, adtype, None, stream)
        return Y
