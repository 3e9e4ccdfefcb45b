"""ctypes binding of include/dq4_int8.h: argument marshalling only, as in _binding.

Layers with 8-bit weights: the row quantizer of LLM.int8 with its outlier columns, the 8-bit
product, the gradient of its input, and a mixture-of-experts layer for few tokens.  Everything is
asynchronous on ``stream`` (default: the current one): nothing here waits for the GPU.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from ._attention import _COUNTERS, _HALF, _bad, _flat, _stream, _stream_of, _workspace
from ._binding import _DTYPE_CODE, Dq4Error, _call_lock, get_lib

# bytes of a new workspace that have to be zero (None: all of them)
_COUNTERS.update({"int8 quantize": None, "int8 linear": 0, "int8 backward": 0, "int8 moe": 0})

_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        L = get_lib()
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        L.dq4_int8_quantize.argtypes = [p, i64, i32, i64, i64, f32, p, p, p, i32, p, p, p, i64, p]
        L.dq4_int8_quantize.restype = ctypes.c_int
        L.dq4_int8_quantize_workspace_bytes.argtypes = [i64]
        L.dq4_int8_quantize_workspace_bytes.restype = i64
        L.dq4_int8_linear.argtypes = [p, p, p, p, i64, i64, i64, p, i32, p, i32, p, i32, p, p, i64,
                                      p, p]
        L.dq4_int8_linear.restype = ctypes.c_int
        L.dq4_int8_linear_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.dq4_int8_linear_workspace_bytes.restype = i64
        L.dq4_int8_linear_backward.argtypes = [p, i32, p, p, i64, i64, i64, p, p, i64, p, p]
        L.dq4_int8_linear_backward.restype = ctypes.c_int
        L.dq4_int8_linear_backward_workspace_bytes.argtypes = [i64, i64, i64]
        L.dq4_int8_linear_backward_workspace_bytes.restype = i64
        L.dq4_int8_moe.argtypes = [p, i64, i32, i64, i64, i64, i64, p, i32, i32, p, p, p, p, p, p,
                                   p, p, i64, p, p]
        L.dq4_int8_moe.restype = ctypes.c_int
        L.dq4_int8_moe_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.dq4_int8_moe_workspace_bytes.restype = i64
        _LIB = L
    return _LIB


# Workspace sizes depend on shapes (and, for the products, the SMs of the current device, which is
# the one of `index`) alone; a device that could not be asked (a negative answer) is not remembered.
@functools.lru_cache(maxsize=256)
def _need_of(index: int, name: str, *shape) -> int:
    need = getattr(_lib(), f"dq4_int8_{name}_workspace_bytes")(*shape)
    if need < 0:
        raise Dq4Error(-need, f"dq4_int8_{name}_workspace_bytes")
    return need


_current_device = torch._C._cuda_getDevice


def _on_gpu(t: torch.Tensor, name: str) -> None:
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (the library reads device memory)")


def _rows(t: torch.Tensor, name: str) -> None:
    """A matrix of rows: any stride between them, a row's values contiguous."""
    _on_gpu(t, name)
    if t.dtype not in _HALF:
        raise TypeError(f"{name}: must be float16 or bfloat16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name}: must be 2-D, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")


def _shape(t: torch.Tensor, name: str, shape) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _weight(CB: torch.Tensor, SCB: torch.Tensor, like: torch.Tensor, name: str, dims: int) -> None:
    """A weight's codes and scales."""
    if CB.dim() != dims:
        raise ValueError(f"{name}: must be {dims}-D, got {tuple(CB.shape)}")
    _shape(SCB, f"{name}'s scales", CB.shape[:-1])
    _flat(CB, name, torch.int8, 0, like)
    _flat(SCB, f"{name}'s scales", torch.float32, 0, like)


# ------------------------------------------------------------- rows in 8 bits
class Int8Rows(NamedTuple):
    """Activations in 8 bits: a value is codes * scales[:, None] / 127, but for the columns
    ``cols``, whose values are ``outliers``.

    ``codes`` int8 [M, K], ``scales`` float32 [M]; ``cols`` int64 [L] (ascending, -1 for none),
    ``outliers`` float16 or bfloat16 [M, L] and ``count`` int32 [1] are None without outlier
    columns.
    """

    codes: torch.Tensor
    scales: torch.Tensor
    cols: Optional[torch.Tensor] = None
    outliers: Optional[torch.Tensor] = None
    count: Optional[torch.Tensor] = None


@functools.lru_cache(maxsize=64)
def _threshold(threshold: float) -> float:
    """The least FP32 number that is not below the threshold: what 16-bit values are at or above of
    one are so of the other, and a threshold above 0 stays one."""
    if threshold < 0:
        return -1.0  # (refused by the library, which would take some of them for 0)
    near = ctypes.c_float(threshold)
    if not near.value < threshold:
        return near.value
    bits = ctypes.c_uint32.from_buffer(near)  # (towards 0 from a positive number: the next)
    bits.value += 1
    return near.value


def int8_quantize(X: torch.Tensor, threshold: float = 0.0, max_outliers: int = 64,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> Int8Rows:
    """Rows of X (M x K, float16 or bfloat16, any row stride) in 8 bits, as LLM.int8 has them.

    A row's scale is its largest magnitude below ``threshold`` (0: of all values).  Columns with
    a value at or above the threshold are outliers: the first ``max_outliers`` of them (1 .. 128)
    have codes of 0 and their values in ``outliers``; ``count`` says how many there are, and
    those past the maximum keep codes that end at +-127.  ``cols`` is what
    :func:`int8_correction_prep` takes, ``outliers`` its subA.  A row with a NaN has a scale of
    NaN.  ``workspace`` (uint8, zero-filled before its first use) is needed with a threshold; by
    default a cached buffer per (device, stream) is used, and in ``torch.cuda.graph`` memory of
    the graph's own.
    """
    if not (X.is_cuda and X.dtype in _HALF and X.dim() == 2 and X.stride(1) == 1):
        _rows(X, "X")
    M, K = X.shape
    index, device = X.get_device(), X.device  # (a device by its index takes torch.empty 2 us more)
    if index != _current_device():
        with torch.cuda.device(index):
            return int8_quantize(X, threshold, max_outliers, workspace, stream)
    handle = _stream(stream, index)
    codes = torch.empty((M, K), dtype=torch.int8, device=device)
    scales = torch.empty(M, dtype=torch.float32, device=device)
    if threshold == 0:
        st = _lib().dq4_int8_quantize(X.data_ptr(), X.stride(0), _DTYPE_CODE[X.dtype], M, K, 0.0,
                                      codes.data_ptr(), scales.data_ptr(), None, 0, None, None,
                                      None, 0, handle)
        if st:
            raise Dq4Error(st, "dq4_int8_quantize")
        return Int8Rows(codes, scales)
    if not 1 <= max_outliers <= 128:
        raise ValueError(f"max_outliers must be 1 .. 128, got {max_outliers}")
    cols = torch.empty(max_outliers, dtype=torch.int64, device=device)
    outliers = torch.empty((M, max_outliers), dtype=X.dtype, device=device)
    count = torch.empty(1, dtype=torch.int32, device=device)
    need = _need_of(index, "quantize", K)
    with _call_lock(index, handle):
        ws_ptr, ws_bytes = _scratch(workspace, need, "int8 quantize", X, handle)
        st = _lib().dq4_int8_quantize(X.data_ptr(), X.stride(0), _DTYPE_CODE[X.dtype], M, K,
                                      _threshold(float(threshold)), codes.data_ptr(),
                                      scales.data_ptr(), cols.data_ptr(), max_outliers,
                                      outliers.data_ptr(),
                                      count.data_ptr(), ws_ptr, ws_bytes, handle)
    if st:
        raise Dq4Error(st, "dq4_int8_quantize")
    return Int8Rows(codes, scales, cols, outliers, count)


# ------------------------------------------------------------- the product
def int8_linear(X: Int8Rows, CB: torch.Tensor, SCB: torch.Tensor,
                bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float16,
                Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                bad: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X W^T + bias with rows X in 8 bits (:func:`int8_quantize`) and W (N x K) in 8 bits:
    CB int8 codes, SCB float32 scales of its rows, a value CB * SCB / 127.

    Outlier columns of X multiply W's values as the 16-bit numbers they are.  ``bias`` ([N]) and
    Y are of ``out_dtype`` (float16, bfloat16 or float32).  K must be a multiple of 16.
    ``workspace`` (uint8) holds X in 16 bits and partial sums; by default a cached buffer per
    (device, stream) is used, and in ``torch.cuda.graph`` memory of the graph's own.  ``bad``
    (int32) counts columns that cannot be used, and waits inside a kernel that ran out, after which
    Y is not to be used.
    """
    codes, scales, cols, outliers, _ = X
    M, K = codes.shape if codes.dim() == 2 else (-1, -1)
    N = CB.shape[0] if CB.dim() == 2 else -1
    index = codes.get_device()
    # (a call of few rows is the host's: first the short way that valid arguments pass)
    if not (codes.is_cuda and CB.is_cuda and codes.dtype is torch.int8 and CB.dtype is torch.int8
            and codes.is_contiguous() and CB.is_contiguous() and CB.get_device() == index
            and scales.shape == (M,) and SCB.shape == (N,) and CB.shape[1] == K
            and scales.dtype is torch.float32 and SCB.dtype is torch.float32
            and scales.is_contiguous() and SCB.is_contiguous()
            and scales.get_device() == index and SCB.get_device() == index):
        _on_gpu(codes, "codes")
        if M < 0 or N < 0 or CB.shape[1] != K:
            raise ValueError(f"codes {tuple(codes.shape)} do not go with CB {tuple(CB.shape)}")
        _flat(codes, "codes", torch.int8, 0, codes)
        _shape(scales, "scales", (M,))
        _flat(scales, "scales", torch.float32, 0, codes)
        _weight(CB, SCB, codes, "CB", 2)
    if index != _current_device():
        with torch.cuda.device(index):
            return int8_linear(X, CB, SCB, bias, out_dtype, Y, workspace, bad, stream)
    if Y is not None:
        out_dtype = Y.dtype
    kind = _DTYPE_CODE.get(out_dtype)
    if kind is None:
        raise TypeError(f"out_dtype: unsupported {out_dtype}")
    cols_ptr = outliers_ptr = bias_ptr = bad_ptr = None
    L = outlier_kind = 0
    if (cols is None) != (outliers is None):
        raise ValueError("cols and outliers come together")
    if cols is not None:
        if cols.dim() != 1 or cols.numel() > 128:
            raise ValueError(f"cols: must be 1-D, 128 at most, got {tuple(cols.shape)}")
        L = cols.numel()
        if outliers.dtype not in _HALF:
            raise TypeError(f"outliers: must be float16 or bfloat16, got {outliers.dtype}")
        _shape(outliers, "outliers", (M, L))
        outlier_kind = _DTYPE_CODE[outliers.dtype]
        cols_ptr = _flat(cols, "cols", torch.int64, 0, codes)
        outliers_ptr = _flat(outliers, "outliers", outliers.dtype, 0, codes)
    if bias is not None:
        _shape(bias, "bias", (N,))
        bias_ptr = _flat(bias, "bias", out_dtype, 0, codes)
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=codes.device)
    else:
        _shape(Y, "Y", (M, N))
        _flat(Y, "Y", out_dtype, 0, codes)
    if bad is not None:
        bad_ptr = _bad(bad, codes)
    handle = _stream(stream, index)
    need = _need_of(index, "linear", M, N, K, L)
    if need == 0 and workspace is None:  # one launch
        st = _lib().dq4_int8_linear(codes.data_ptr(), scales.data_ptr(), CB.data_ptr(),
                                    SCB.data_ptr(), M, N, K, cols_ptr, L, outliers_ptr,
                                    outlier_kind, bias_ptr, kind, Y.data_ptr(), None, 0, bad_ptr,
                                    handle)
    else:
        with _call_lock(index, handle):
            ws_ptr, ws_bytes = _scratch(workspace, need, "int8 linear", codes, handle)
            st = _lib().dq4_int8_linear(codes.data_ptr(), scales.data_ptr(), CB.data_ptr(),
                                        SCB.data_ptr(), M, N, K, cols_ptr, L, outliers_ptr,
                                        outlier_kind, bias_ptr, kind, Y.data_ptr(), ws_ptr,
                                        ws_bytes, bad_ptr, handle)
    if st:
        raise Dq4Error(st, "dq4_int8_linear")
    return Y


def _scratch(workspace, need: int, what: str, like: torch.Tensor, handle):
    """Address and size of the call's workspace; none if it needs none."""
    if need == 0 and workspace is None:
        return None, 0
    ws = _workspace(workspace, need, what, like, handle)
    return ws.data_ptr(), ws.numel()


def int8_linear_backward(dY: torch.Tensor, CB: torch.Tensor, SCB: torch.Tensor,
                         dX: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         bad: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dX = dY W: the gradient of :func:`int8_linear`'s input, its rounding to 8 bits taken as
    the identity.

    dY is M x N (float16 or bfloat16, contiguous); W's values are rounded to its type, as
    :func:`int8_correction_prep` has them.  N must be a multiple of 8, K of 16.  ``workspace``
    (of partial sums) and ``bad`` as for :func:`int8_linear`.
    """
    index = dY.get_device()
    # (first the short way that valid arguments pass, as in int8_linear)
    if not (dY.is_cuda and CB.is_cuda and dY.dtype in _HALF and CB.dtype is torch.int8
            and SCB.dtype is torch.float32 and dY.dim() == 2 and CB.dim() == 2
            and CB.shape[0] == dY.shape[1] and SCB.shape == CB.shape[:1]
            and dY.is_contiguous() and CB.is_contiguous() and SCB.is_contiguous()
            and CB.get_device() == index and SCB.get_device() == index):
        _on_gpu(dY, "dY")
        if dY.dtype not in _HALF:
            raise TypeError(f"dY: must be float16 or bfloat16, got {dY.dtype}")
        if dY.dim() != 2 or CB.dim() != 2 or dY.shape[1] != CB.shape[0]:
            raise ValueError(f"dY {tuple(dY.shape)} does not go with CB {tuple(CB.shape)}")
        _flat(dY, "dY", dY.dtype, 0, dY)
        _weight(CB, SCB, dY, "CB", 2)
    if index != _current_device():
        with torch.cuda.device(index):
            return int8_linear_backward(dY, CB, SCB, dX, workspace, bad, stream)
    M, N = dY.shape
    K = CB.shape[1]
    if dX is None:
        dX = torch.empty((M, K), dtype=dY.dtype, device=dY.device)
    else:
        _shape(dX, "dX", (M, K))
        _flat(dX, "dX", dY.dtype, 0, dY)
    bad_ptr = None if bad is None else _bad(bad, dY)
    handle = _stream(stream, index)
    need = _need_of(index, "linear_backward", M, N, K)
    with _call_lock(index, handle):
        ws_ptr, ws_bytes = _scratch(workspace, need, "int8 backward", dY, handle)
        st = _lib().dq4_int8_linear_backward(dY.data_ptr(), _DTYPE_CODE[dY.dtype], CB.data_ptr(),
                                             SCB.data_ptr(), M, N, K, dX.data_ptr(), ws_ptr,
                                             ws_bytes, bad_ptr, handle)
    if st:
        raise Dq4Error(st, "dq4_int8_linear_backward")
    return dX


# ------------------------------------------------------------- mixture of experts
def _routing(T: int, top_k: int, like: torch.Tensor):
    return (torch.empty((T, top_k), dtype=torch.int32, device=like.device),
            torch.empty((T, top_k), dtype=torch.float32, device=like.device))


def int8_moe(X: torch.Tensor, logits: torch.Tensor, w1: torch.Tensor, s1: torch.Tensor,
             w2: torch.Tensor, s2: torch.Tensor, top_k: int, renormalize: bool = True,
             return_routing: bool = False, workspace: Optional[torch.Tensor] = None,
             bad: Optional[torch.Tensor] = None, stream=None):
    """A mixture-of-experts layer for few tokens (256 at most) over 8-bit weights.

    X is T x H (float16 or bfloat16, its rows 16-byte aligned), ``logits`` T x E (float32).  Each
    token goes through the ``top_k`` experts (16 at most) with its largest logits, the lower index
    first where they are equal, weighted by their softmax over the chosen ones (``renormalize``) or
    over all:
    ``y = sum p_e W2_e (silu(Wg_e x) * (Wu_e x))``.  ``w1`` int8 [E, 2 I, H] holds the rows of
    Wg, then those of Wu, ``w2`` int8 [E, H, I]; ``s1`` [E, 2 I] and ``s2`` [E, H] are float32
    scales of their rows, a value w * s / 127.  H and I are multiples of 16, and not 0 with tokens.
    Returns Y (T x H, X's dtype), or (Y, ids, weights) with the choices, int32 and float32
    [T, top_k].
    ``workspace`` (uint8) holds the rows between the launches; by default a cached buffer per
    (device, stream) is used, and in ``torch.cuda.graph`` memory of the graph's own.  ``bad``
    (int32) counts waits inside a kernel that ran out, after which Y is not to be used.
    """
    index = X.get_device()
    T, H = X.shape if X.dim() == 2 else (-1, -1)
    E, I = (w1.shape[0], w2.shape[2]) if w1.dim() == 3 and w2.dim() == 3 else (-1, -1)
    # (first the short way that valid arguments pass, as in int8_linear)
    if not (X.is_cuda and X.dtype in _HALF and T >= 0 and E >= 0 and X.stride(1) == 1
            and w1.shape == (E, 2 * I, H) and w2.shape == (E, H, I) and s1.shape == (E, 2 * I)
            and s2.shape == (E, H) and logits.shape == (T, E) and w1.dtype is torch.int8
            and w2.dtype is torch.int8 and s1.dtype is torch.float32
            and s2.dtype is torch.float32 and logits.dtype is torch.float32
            and w1.is_contiguous() and w2.is_contiguous() and s1.is_contiguous()
            and s2.is_contiguous() and logits.is_contiguous() and w1.get_device() == index
            and w2.get_device() == index and s1.get_device() == index
            and s2.get_device() == index and logits.get_device() == index):
        _rows(X, "X")
        _weight(w1, s1, X, "w1", 3)
        _weight(w2, s2, X, "w2", 3)
        _shape(w1, "w1", (E, 2 * I, H))
        _shape(w2, "w2", (E, H, I))
        _shape(logits, "logits", (T, E))
        _flat(logits, "logits", torch.float32, 0, X)
    if index != _current_device():
        with torch.cuda.device(index):
            return int8_moe(X, logits, w1, s1, w2, s2, top_k, renormalize, return_routing,
                            workspace, bad, stream)
    if not 1 <= top_k <= min(E, 16):
        raise ValueError(f"top_k must be 1 .. {min(E, 16)}, got {top_k}")
    bad_ptr = None if bad is None else _bad(bad, X)
    handle = _stream(stream, index)
    Y = torch.empty((T, H), dtype=X.dtype, device=X.device)
    if return_routing or handle == torch._C._cuda_getCurrentRawStream(index):
        ids, weights = _routing(T, top_k, X)
    else:  # nobody else holds them: memory of the stream that uses them, which is given back to it
        with torch.cuda.stream(_stream_of(handle, index)):
            ids, weights = _routing(T, top_k, X)
    need = _need_of(index, "moe", T, H, I, top_k)
    with _call_lock(index, handle):
        ws_ptr, ws_bytes = _scratch(workspace, need, "int8 moe", X, handle)
        st = _lib().dq4_int8_moe(X.data_ptr(), X.stride(0), _DTYPE_CODE[X.dtype], T, H, I, E,
                                 logits.data_ptr(), top_k, renormalize, w1.data_ptr(),
                                 s1.data_ptr(), w2.data_ptr(), s2.data_ptr(), ids.data_ptr(),
                                 weights.data_ptr(), Y.data_ptr(), ws_ptr, ws_bytes, bad_ptr,
                                 handle)
    if st:
        raise Dq4Error(st, "dq4_int8_moe")
    return (Y, ids, weights) if return_routing else Y
