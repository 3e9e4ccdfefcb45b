"""ctypes binding of include/dq4_attn.h: argument marshalling only, as in _binding.

The attention around the 4-bit projections: the norm of queries and keys with the position
rotation (forward and backward), the append to a paged 8-bit key/value cache, and the attention
that reads it.  Everything is asynchronous on ``stream`` (default: the current one) and reads
lengths, pages and positions on the device: nothing here waits for the GPU.
"""

from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from ._binding import _DTYPE_CODE, Dq4Error, _call_lock, _check, _stream_handle, get_lib

_HALF = (torch.float16, torch.bfloat16)
PAGE_TOKENS = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128)
_INT_MAX = 2 ** 31 - 1


class _Cache(ctypes.Structure):
    """dq4_kv8_cache of dq4_attn.h."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int32), ("page", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        L = get_lib()
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        L.dq4_qk_norm_rope.argtypes = [p, i64, i64, p, i64, i64, i32, i64, i32, i32, i32, p, p,
                                       f32, p, p, i64, i32, i32, p, p, p, p, p]
        L.dq4_qk_norm_rope.restype = ctypes.c_int
        L.dq4_qk_norm_rope_backward.argtypes = [p, p, p, i64, i64, p, i64, i64, i32, i64, i32,
                                                i32, i32, p, p, f32, p, p, i64, i32, i32, p, p,
                                                p, p, p, p, i64, p, p]
        L.dq4_qk_norm_rope_backward.restype = ctypes.c_int
        L.dq4_qk_norm_rope_backward_workspace_bytes.argtypes = [i32]
        L.dq4_qk_norm_rope_backward_workspace_bytes.restype = i64
        L.dq4_kv8_append.argtypes = [p, p, i64, i64, p, i64, i64, i32, i64, p, i64, i32, p, p,
                                     i64, p, p, i64, i32, i32, p, p]
        L.dq4_kv8_append.restype = ctypes.c_int
        L.dq4_kv8_attention.argtypes = [p, p, i64, i64, i32, i64, i32, p, i64, i32, p, p, i64,
                                        i32, f32, i32, i32, p, p, p, i64, p, p]
        L.dq4_kv8_attention.restype = ctypes.c_int
        L.dq4_kv8_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32]
        L.dq4_kv8_attention_workspace_bytes.restype = i64
        _LIB = L
    return _LIB


# ------------------------------------------------------------- helpers
# A call of few tokens is bound by the host, so the checks below first take the short way that a
# valid argument passes, and look for what is wrong only if it does not.
_WORKSPACES = {}
_COUNTERS = {"attention": 2048, "norm": 256}  # bytes that have to be zero at first, at the head


def _workspace(workspace, need: int, what: str, like: torch.Tensor, handle) -> torch.Tensor:
    """The caller's workspace, or the stream's (_stream_workspace).  Memory of the latter comes from
    the stream that uses it."""
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, need, like.device)
        return workspace
    index = like.get_device()
    if handle == torch._C._cuda_getCurrentRawStream(index):
        return _stream_workspace(need, what, like, index, handle)
    stream = (torch.cuda.ExternalStream(handle, index) if handle else
              torch.cuda.default_stream(index))
    with torch.cuda.stream(stream):
        return _stream_workspace(need, what, like, index, handle)


def _stream_workspace(need: int, what: str, like: torch.Tensor, index: int, handle):
    """The cached zero-filled workspace of (operator, device, current stream), grown to `need`
    bytes, and to twice its size at least.  In a capture: one of the graph's own memory, whose
    counters the graph itself clears, so that its replays share nothing with other calls."""
    if torch._C._cuda_isCurrentStreamCapturing():
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
        ws[:_COUNTERS[what]].zero_()
        return ws
    key = (what, index, handle)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < need:
        if ws is not None:
            need = max(need, 2 * ws.numel())
        ws = torch.zeros(max(need, 1), dtype=torch.uint8, device=like.device)
        _WORKSPACES[key] = ws
    return ws


def _stream(stream, index: int) -> int:
    """The handle of `stream`, or of the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return _stream_handle(stream, None)


def _flat(t: torch.Tensor, name: str, dtype, numel: int, like: torch.Tensor) -> int:
    """The address of a contiguous tensor of `dtype` with `numel` elements at least, on like's
    device."""
    if (t.dtype is not dtype or t.get_device() != like.get_device() or t.numel() < numel
            or not t.is_contiguous()):
        _check(t, name, dtype, numel, like.device)
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, dtype, like: torch.Tensor) -> None:
    """A tokens x heads x head_dim tensor: any strides, but a head's values contiguous."""
    if (t.is_cuda and t.dtype is dtype and t.get_device() == like.get_device() and t.dim() == 3
            and t.stride(2) == 1):
        return
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (the library reads device memory)")
    if t.device != like.device:
        raise ValueError(f"{name}: expected a tensor on {like.device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name}: must be tokens x heads x head_dim, got {tuple(t.shape)}")
    if t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name}: the values of a head must be contiguous")


def _output(out, name: str, shape, like: torch.Tensor) -> torch.Tensor:
    """`out` if given, else a new tensor; contiguous, of like's type."""
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if tuple(out.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(out.shape)}")
    _flat(out, name, like.dtype, 0, like)
    return out


def _bad(bad, like) -> Optional[int]:
    return None if bad is None else _flat(bad, "bad", torch.int32, 1, like)


_NO_ROWS = 256  # an address: empty tensors have none, and none means no rotation


def _tables(cos, sin, like) -> Tuple[Optional[int], Optional[int], int, int]:
    """(cos, sin, rows, rotary) of the rotation's tables."""
    if cos is None and sin is None:
        return None, None, 0, 0
    if cos is None or sin is None:
        raise ValueError("cos and sin come together")
    if cos.dim() != 2 or cos.shape != sin.shape:
        raise ValueError(f"cos and sin must be positions x rotary / 2 and alike, got "
                         f"{tuple(cos.shape)} and {tuple(sin.shape)}")
    rows, half = cos.shape
    c, s = (_flat(t, n, torch.float32, 0, like) for t, n in ((cos, "cos"), (sin, "sin")))
    if rows == 0 and half > 0:  # tables all the same, with no position in them: never followed
        c = s = _NO_ROWS
    return c, s, rows, 2 * half


# ------------------------------------------------------------- norm and rotation
def _norm_args(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
    """Checked arguments of the C entry points, from q to positions."""
    dtype = q.dtype
    if dtype not in _DTYPE_CODE:
        raise TypeError(f"q: unsupported dtype {dtype}")
    _heads(q, "q", dtype, q)
    tokens, hq, dim = q.shape
    qs = q.stride()
    qw = kw = k_ptr = pos = None
    hk, ks = 0, (0, 0)
    if k is not None:
        _heads(k, "k", dtype, q)
        k_tokens, hk, k_dim = k.shape
        if k_tokens != tokens or k_dim != dim:
            raise ValueError(f"k {tuple(k.shape)} does not go with q {tuple(q.shape)}")
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight come together")
        k_ptr, ks = k.data_ptr(), k.stride()
    if q_weight is not None:
        qw = _flat(q_weight, "q_weight", dtype, dim, q)
        if k is not None:
            kw = _flat(k_weight, "k_weight", dtype, dim, q)
    tables = _tables(cos, sin, q)
    if cos is not None:
        if positions is None:
            raise ValueError("positions: needed with cos and sin")
        pos = _flat(positions, "positions", torch.int64, tokens, q)
    return (q.data_ptr(), qs[0], qs[1], k_ptr, ks[0], ks[1], _DTYPE_CODE[dtype], tokens, hq, hk,
            dim, qw, kw, eps, *tables, interleaved, pos)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                 k_weight: Optional[torch.Tensor], cos: Optional[torch.Tensor] = None,
                 sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 bad: Optional[torch.Tensor] = None, stream=None):
    """Norm and rotation of every head of q and k in one launch; returns (q_out, k_out).

    ``y = R(positions[t]) (w * x / sqrt(mean(x^2) + eps))`` for q (tokens x heads x head_dim)
    and k (tokens x kv_heads x head_dim, or None), float16, bfloat16 or float32, with any
    strides between tokens and heads (views of a fused projection).  Without weights there is
    no norm; without ``cos`` and ``sin`` (float32 tables, positions x rotary / 2) no rotation.
    ``interleaved`` pairs values 2i and 2i + 1, else i and i + rotary / 2.  A position outside
    the tables yields zeros, counted into ``bad`` (int32) for each head.
    """
    args = _norm_args(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    q_out = _output(q_out, "q_out", tuple(q.shape), q)
    k_ptr = None
    if k is not None:
        k_out = _output(k_out, "k_out", tuple(k.shape), q)
        k_ptr = k_out.data_ptr()
    st = _lib().dq4_qk_norm_rope(*args, q_out.data_ptr(), k_ptr, _bad(bad, q),
                                 _stream(stream, q.get_device()))
    if st:
        raise Dq4Error(st, "dq4_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor],
                          q: torch.Tensor, k: Optional[torch.Tensor],
                          q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                          cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
                          positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          interleaved: bool = False, dq: Optional[torch.Tensor] = None,
                          dk: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          bad: Optional[torch.Tensor] = None, stream=None):
    """The gradients of :func:`qk_norm_rope`: (dq, dk, dq_weight, dk_weight).

    ``dq_out`` and ``dk_out`` are the outputs' gradients (contiguous, q's dtype); the weights'
    gradients are float32 (None without weights), summed in a fixed order.  ``workspace``
    (uint8, zero-filled before its first use) holds partial sums; by default a cached buffer
    per (device, stream) is used, and in ``torch.cuda.graph`` memory of the graph's own (a
    workspace that is given belongs to one call or replay at a time).
    """
    args = _norm_args(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    dim = q.shape[2]
    dq_out_ptr = _flat(dq_out, "dq_out", q.dtype, q.numel(), q)
    dq = _output(dq, "dq", tuple(q.shape), q)
    dk_out_ptr = dk_ptr = dqw = dkw = dkw_ptr = None
    if k is not None:
        if dk_out is None:
            raise ValueError("dk_out: needed with k")
        dk_out_ptr = _flat(dk_out, "dk_out", q.dtype, k.numel(), q)
        dk = _output(dk, "dk", tuple(k.shape), q)
        dk_ptr = dk.data_ptr()
    bad_ptr = _bad(bad, q)
    handle = _stream(stream, q.get_device())
    weights = (None, None, None, 0)
    with _call_lock(q.get_device(), handle):
        if q_weight is not None:
            dqw = torch.empty(dim, dtype=torch.float32, device=q.device)
            if k is not None:
                dkw = torch.empty(dim, dtype=torch.float32, device=q.device)
                dkw_ptr = dkw.data_ptr()
            ws = _workspace(workspace, _norm_need(dim), "norm", q, handle)
            weights = (dqw.data_ptr(), dkw_ptr, ws.data_ptr(), ws.numel())
        st = _lib().dq4_qk_norm_rope_backward(dq_out_ptr, dk_out_ptr, *args, dq.data_ptr(),
                                              dk_ptr, *weights, bad_ptr, handle)
    if st:
        raise Dq4Error(st, "dq4_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


@functools.lru_cache(maxsize=64)
def _norm_need(dim: int) -> int:
    return _lib().dq4_qk_norm_rope_backward_workspace_bytes(dim)


# ------------------------------------------------------------- the cache
class KV8Cache:
    """A paged key/value cache in 8 bits: e4m3 codes and one scale for each page and head.

    ``k`` and ``v`` are float8_e4m3fn [pages, kv_heads, page, head_dim], ``k_scale`` and
    ``v_scale`` float32 [pages, kv_heads]; a stored value is code * scale.  Nothing has to be
    initialized: slots and scales are read only where tokens were appended.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        if k.dim() != 4:
            raise ValueError(f"k: must be pages x kv_heads x page x head_dim, got "
                             f"{tuple(k.shape)}")
        pages, heads, page, dim = k.shape
        if heads < 1:
            raise ValueError("k: the cache needs one kv head at least")
        if page not in PAGE_TOKENS:
            raise ValueError(f"k: a page holds {PAGE_TOKENS} tokens, got {page}")
        if dim not in HEAD_DIMS:
            raise ValueError(f"k: head_dim must be one of {HEAD_DIMS}, got {dim}")
        if v.shape != k.shape:
            raise ValueError(f"v: expected shape {tuple(k.shape)}, got {tuple(v.shape)}")
        for t, name in ((k, "k"), (v, "v")):
            _check(t, name, torch.float8_e4m3fn, k.numel(), k.device)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if tuple(t.shape) != (pages, heads):
                raise ValueError(f"{name}: expected shape {(pages, heads)}, got "
                                 f"{tuple(t.shape)}")
            _check(t, name, torch.float32, pages * heads, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_heads, self.page, self.head_dim = heads, page, dim
        self.c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        pages, heads, page, dim)
        self.ref = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page: int, head_dim: int, device="cuda"):
        """A cache of its own tensors."""
        shape = (pages, kv_heads, page, head_dim)
        codes = [torch.empty(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        scales = [torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def _batch(cache, tokens: int, block_table, seq_lens, cu):
    """Checked pointers of the ragged batch: (table, stride, width, lens, cu, sequences)."""
    like = cache.k
    if block_table.dim() != 2:
        raise ValueError(f"block_table: must be sequences x pages, got "
                         f"{tuple(block_table.shape)}")
    seqs, width = block_table.shape
    stride, inner = block_table.stride()
    if (block_table.dtype is not torch.int32 or block_table.get_device() != like.get_device()
            or (width > 1 and inner != 1)):
        raise ValueError(f"block_table: must be int32 rows on {like.device}")
    lens = _flat(seq_lens, "seq_lens", torch.int32, seqs, like)
    if cu is not None:
        cu = _flat(cu, "cu", torch.int32, seqs + 1, like)
    elif tokens != seqs:
        raise ValueError(f"{tokens} tokens for {seqs} sequences: cu says how many each has")
    return block_table.data_ptr(), stride, width, lens, cu, seqs


def kv8_append(cache: KV8Cache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, cu: Optional[torch.Tensor] = None,
               cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
               interleaved: bool = False, bad: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """Append tokens to the cache, keys rotated by their positions on the way; one launch.

    k and v are tokens x kv_heads x head_dim (float16 or bfloat16).  Sequence b's are rows
    ``cu[b] .. cu[b + 1] - 1`` (int32; None: one each), its length with them ``seq_lens[b]``
    (int32), and page ``block_table[b, j]`` (int32) holds its tokens from j * page on.  Scales
    are the least powers of two that fit; a page whose scale grows has its earlier codes
    rescaled.  ``bad`` (int32) counts tokens that have no place.
    """
    if k.dtype not in _HALF:
        raise TypeError("k must be float16 or bfloat16")
    like = cache.k
    _heads(k, "k", k.dtype, like)
    _heads(v, "v", k.dtype, like)
    tokens, heads, dim = k.shape
    if k.shape != v.shape or heads != cache.kv_heads or dim != cache.head_dim:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)}: expected (tokens, "
                         f"{cache.kv_heads}, {cache.head_dim})")
    table, stride, width, lens, cu_ptr, seqs = _batch(cache, tokens, block_table, seq_lens, cu)
    tables = _tables(cos, sin, like)
    ks, vs = k.stride(), v.stride()
    st = _lib().dq4_kv8_append(
        cache.ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], _DTYPE_CODE[k.dtype],
        tokens, table, stride, width, lens, cu_ptr, seqs, *tables, interleaved,
        _bad(bad, like), _stream(stream, like.get_device()))
    if st:
        raise Dq4Error(st, "dq4_kv8_append")


def kv8_attention(cache: KV8Cache, q: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, cu: Optional[torch.Tensor] = None,
                  max_new: Optional[int] = None, scale: Optional[float] = None,
                  causal: bool = True, window: int = 0, out: Optional[torch.Tensor] = None,
                  return_lse: bool = False, workspace: Optional[torch.Tensor] = None,
                  bad: Optional[torch.Tensor] = None, stream=None):
    """Attention of q (tokens x heads x head_dim, float16 or bfloat16) over the cache.

    The batch is given as for :func:`kv8_append`; a token at position p sees its sequence's
    keys j <= p (all of them if not ``causal``) with j > p - window if ``window`` > 0.
    ``scale`` defaults to 1 / sqrt(head_dim); ``max_new`` is the most new tokens of a sequence
    (an estimate will do: it chooses the kernel; default 1, or the mean with ``cu``).  Returns
    ``out`` (tokens x heads x head_dim), or (out, lse) with the float32 log-sums.  A row that
    sees no key gets zeros and -inf.  ``workspace`` (uint8, zero-filled before its first use)
    holds partial results; by default a cached buffer per (device, stream) is used, and in
    ``torch.cuda.graph`` memory of the graph's own, cleared in the graph (1.2 us a call).  A
    workspace that is given belongs to one call, or replay of a captured one, at a time.
    """
    if q.dtype not in _HALF:
        raise TypeError("q must be float16 or bfloat16")
    like = cache.k
    _heads(q, "q", q.dtype, like)
    tokens, heads, dim = q.shape
    if dim != cache.head_dim or heads % cache.kv_heads:
        raise ValueError(f"q {tuple(q.shape)}: the cache has {cache.kv_heads} heads of "
                         f"{cache.head_dim}")
    table, stride, width, lens, cu_ptr, seqs = _batch(cache, tokens, block_table, seq_lens, cu)
    if max_new is None:
        max_new = 1 if cu is None else -(-tokens // max(seqs, 1))
    # (the library takes 32 bits: no sequence is longer)
    window, max_new = max(-1, min(window, _INT_MAX)), max(-1, min(max_new, _INT_MAX))
    out = _output(out, "out", (tokens, heads, dim), q)
    lse = lse_ptr = None
    if return_lse:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=q.device)
        lse_ptr = lse.data_ptr()
    bad_ptr = _bad(bad, like)
    handle = _stream(stream, like.get_device())
    need = _attention_need(tokens, seqs, heads, cache.kv_heads, dim)
    qs = q.stride()
    with _call_lock(like.get_device(), handle):
        ws = _workspace(workspace, need, "attention", like, handle)
        st = _lib().dq4_kv8_attention(
            cache.ref, q.data_ptr(), qs[0], qs[1], _DTYPE_CODE[q.dtype], tokens, heads, table,
            stride, width, lens, cu_ptr, seqs, max_new,
            1 / math.sqrt(dim) if scale is None else scale, causal, window, out.data_ptr(),
            lse_ptr, ws.data_ptr(), ws.numel(), bad_ptr, handle)
    if st:
        raise Dq4Error(st, "dq4_kv8_attention")
    return (out, lse) if return_lse else out


@functools.lru_cache(maxsize=256)
def _attention_need(tokens: int, seqs: int, heads: int, kv_heads: int, dim: int) -> int:
    return _lib().dq4_kv8_attention_workspace_bytes(tokens, seqs, heads, kv_heads, dim)
