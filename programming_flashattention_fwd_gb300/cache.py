"""Operators of a paged key/value cache: argument marshalling over libfa_gb300.so.

``KVCache`` names the tensors of one layer's cache; ``tree_attention`` attends drafted tokens over
it, ``cache_append`` writes accepted tokens, ``cache_weights`` adds up the attention that each slot
receives and ``cache_evict`` shrinks the cache by it.  include/fa.h defines each operator; as in
``binding``, every step of the computation runs in the library's CUDA kernels and a non-zero
status raises ``FaError``.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from .binding import FaError, _check_stream_device, _OnDevice, _stream_handle, fa_strerror, load_library

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class _CacheStruct(ctypes.Structure):
    """fa_cache_t of include/fa.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("seq_len", ctypes.c_void_p), ("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("page", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("dtype", ctypes.c_int)]


_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_CP = ctypes.POINTER(_CacheStruct)
_SIGNATURES = {
    "fa_tree_workspace_bytes": (_Z, [_I] * 4),
    "fa_tree_fwd": (_I, [_CP] + [_P] * 7 + [_I, _I, _F, _P, _Z, _P]),
    "fa_cache_append": (_I, [_CP] + [_P] * 7 + [_I, _P]),
    "fa_weights_workspace_bytes": (_Z, []),
    "fa_cache_weights": (_I, [_CP] + [_P] * 6 + [_I, _I, _I, _F, _P, _Z, _P]),
    "fa_evict_workspace_bytes": (_Z, [_I] * 4),
    "fa_cache_evict": (_I, [_CP] + [_P] * 6 + [_I, _I, _I, _P, _Z, _P]),
}
_lib = None


def _library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = load_library()
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


def _run(st: int) -> None:
    if st != 0:
        raise FaError(st, fa_strerror(st))


def _need(name: str, t, shape, dtype, device) -> int:
    """The address of a dense CUDA tensor of this shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device} but the cache is on {device}: "
                         "every tensor of one call must be on the same GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _maybe(name: str, t, shape, dtype, device) -> Optional[int]:
    return None if t is None else _need(name, t, shape, dtype, device)


def _keep_for(t: torch.Tensor, stream) -> None:
    """A temporary used on `stream` must not be reused by the current stream's later work before it is done."""
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=t.device)
        t.record_stream(s)


class KVCache:
    """The keys and values of B sequences in pages (fa_cache_t).

    k, v     [num_pages, Hkv, page, D] bf16 or fp16, contiguous CUDA tensors; page a multiple of 16
    seq_len  [B] int32: slots in use of each sequence, read by the kernels when they run
    table    [B, max_pages] int32: the page of each run of `page` slots; None for a dense cache,
             whose pages belong to the sequences in order (num_pages // B each)

    Holds references to the tensors and no state of its own: update seq_len and table in place.
    """
    __slots__ = ("k", "v", "seq_len", "table", "device", "dtype", "B", "Hkv", "D", "page", "capacity", "_c", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, seq_len: torch.Tensor, table: Optional[torch.Tensor] = None):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a [num_pages, Hkv, page, D] tensor")
        if k.dtype not in _DTYPES:
            raise ValueError(f"a cache is bf16 or fp16, not {k.dtype}")
        if not k.is_cuda:
            raise ValueError("k must be a CUDA tensor")
        dev, dt = k.device, k.dtype
        num, Hkv, page, D = k.shape
        if not isinstance(seq_len, torch.Tensor) or seq_len.dim() != 1:
            raise ValueError("seq_len must be a [B] tensor")
        B = seq_len.shape[0]
        if table is None:
            per = num // B if B else 0
        else:
            if not isinstance(table, torch.Tensor) or table.dim() != 2:
                raise ValueError("table must be a [B, max_pages] tensor")
            per = table.shape[1]
        self._c = _CacheStruct(_need("k", k, k.shape, dt, dev), _need("v", v, k.shape, dt, dev),
                               _maybe("table", table, (B, per), torch.int32, dev),
                               _need("seq_len", seq_len, (B,), torch.int32, dev), B, Hkv, D, page, per, num, _DTYPES[dt])
        self._ref = ctypes.pointer(self._c)
        self.k, self.v, self.seq_len, self.table = k, v, seq_len, table
        self.device, self.dtype, self.B, self.Hkv, self.D, self.page = dev, dt, B, Hkv, D, page
        self.capacity = per * page


def tree_workspace_bytes(Hq: int, Hkv: int, T: int, D: int) -> int:
    """Bytes of the workspace of ``tree_attention`` for T drafted tokens."""
    return _library().fa_tree_workspace_bytes(Hq, Hkv, T, D)


def _workspace(need: int, given: Optional[torch.Tensor], device, stream) -> Tuple[torch.Tensor, int]:
    if given is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
        _keep_for(ws, stream)
        return ws, need
    if not given.is_cuda or given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the cache's device")
    return given, given.numel() * given.element_size()


def tree_attention(q, k_new, v_new, cache: KVCache, parent=None, draft_len=None, scale: Optional[float] = None,
                   o=None, lse=None, workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of drafted tokens over the cache and over the drafted tokens on their path (fa_tree_fwd).

    q [B, Hq, T, D], k_new and v_new [B, Hkv, T, D] in the cache's type; parent [B, T] int32 (-1: a
    root; None: a chain), draft_len [B] int32 (None: T).  Returns (o [B, Hq, T, D], lse [B, Hq, T]
    float32), in o and lse where they are given; rows at or behind draft_len are not written.
    scale defaults to D ** -0.5.  workspace: tree_workspace_bytes(...) bytes that no other call in
    flight uses; allocated when None."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, Hq, T, D] tensor")
    dev, dt = cache.device, cache.dtype
    B, Hq, T, D = q.shape
    if B != cache.B or D != cache.D:
        raise ValueError(f"q must have the cache's {cache.B} sequences and head dimension {cache.D}")
    new = (B, cache.Hkv, T, D)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
    lib = _library()
    args = (_need("q", q, q.shape, dt, dev), _need("k_new", k_new, new, dt, dev), _need("v_new", v_new, new, dt, dev),
            _maybe("parent", parent, (B, T), torch.int32, dev), _maybe("draft_len", draft_len, (B,), torch.int32, dev),
            _need("o", o, q.shape, dt, dev), _need("lse", lse, (B, Hq, T), torch.float32, dev))
    _check_stream_device(stream, dev)
    ws, size = _workspace(lib.fa_tree_workspace_bytes(Hq, cache.Hkv, T, D), workspace, dev, stream)
    with _OnDevice(dev):
        _run(lib.fa_tree_fwd(cache._ref, *args, Hq, T, 1.0 / math.sqrt(D) if scale is None else scale, ws.data_ptr(), size,
                             _stream_handle(stream)))
    return o, lse


def cache_append(cache: KVCache, k_new, v_new, path=None, count=None, weight=None, pos=None, start=None,
                 stream=None) -> None:
    """Writes tokens behind the slots in use (fa_cache_append): slot seq_len[b] + i takes token path[b, i]
    (token i without a path) of k_new, v_new [B, Hkv, T, D], i < count[b] (None: T).  weight
    [B, Hkv, capacity] float32 becomes 0 and pos [B, Hkv, capacity] int32 start[b] + i at the new slots,
    where given.  seq_len is not changed: add count to it after the last layer."""
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4:
        raise ValueError("k_new must be a [B, Hkv, T, D] tensor")
    dev, dt, T = cache.device, cache.dtype, k_new.shape[2]
    B = cache.B
    new, slots = (B, cache.Hkv, T, cache.D), (B, cache.Hkv, cache.capacity)
    if path is not None and count is None:
        raise ValueError("a path needs count")
    if pos is not None and start is None:
        raise ValueError("pos needs start")
    args = (_need("k_new", k_new, new, dt, dev), _need("v_new", v_new, new, dt, dev),
            _maybe("path", path, (B, T), torch.int32, dev), _maybe("count", count, (B,), torch.int32, dev),
            _maybe("start", start, (B,), torch.int32, dev), _maybe("weight", weight, slots, torch.float32, dev),
            _maybe("pos", pos, slots, torch.int32, dev))
    _check_stream_device(stream, dev)
    lib = _library()
    with _OnDevice(dev):
        _run(lib.fa_cache_append(cache._ref, *args, T, _stream_handle(stream)))


def weights_workspace_bytes() -> int:
    """Bytes of the workspace of ``cache_weights``."""
    return _library().fa_weights_workspace_bytes()


def cache_weights(cache: KVCache, q, lse, weight=None, path=None, count=None, causal: bool = True,
                  scale: Optional[float] = None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Adds to each slot the attention weight that it receives from the rows of q (fa_cache_weights).

    q [B, Hq, T, D], lse [B, Hq, T] as the attention left it; path [B, T] and count [B] int32 as in
    ``cache_append`` (the accepted rows); causal: row i is the query of slot seq_len[b] - count[b] + i
    and sees the slots up to its own.  weight [B, Hkv, capacity] float32 (None: zeros) is added to; the
    result is written to out, which defaults to weight itself (without a weight, to a new tensor of zeros)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, Hq, T, D] tensor")
    dev = cache.device
    B, Hq, T, D = q.shape
    if B != cache.B or D != cache.D:
        raise ValueError(f"q must have the cache's {cache.B} sequences and head dimension {cache.D}")
    if path is not None and count is None:
        raise ValueError("a path needs count")
    slots = (B, cache.Hkv, cache.capacity)
    if out is None:
        out = torch.zeros(slots, dtype=torch.float32, device=dev) if weight is None else weight
    args = (_need("q", q, q.shape, cache.dtype, dev), _need("lse", lse, (B, Hq, T), torch.float32, dev),
            _maybe("path", path, (B, T), torch.int32, dev), _maybe("count", count, (B,), torch.int32, dev),
            _maybe("weight", weight, slots, torch.float32, dev), _need("out", out, slots, torch.float32, dev))
    _check_stream_device(stream, dev)
    lib = _library()
    ws, size = _workspace(lib.fa_weights_workspace_bytes(), workspace, dev, stream)
    with _OnDevice(dev):
        _run(lib.fa_cache_weights(cache._ref, *args, Hq, T, int(bool(causal)), 1.0 / math.sqrt(D) if scale is None else scale,
                                  ws.data_ptr(), size, _stream_handle(stream)))
    return out


def evict_workspace_bytes(B: int, Hkv: int, capacity: int, keep: int) -> int:
    """Bytes of the workspace of ``cache_evict``."""
    return _library().fa_evict_workspace_bytes(B, Hkv, capacity, keep)


def cache_evict(cache: KVCache, weight, pos, keep: int, first: int = 0, last: int = 0, next_pos=None, weight_out=None,
                pos_out=None, new_len=None, workspace=None, stream=None) -> torch.Tensor:
    """Shrinks every sequence and KV head to `keep` slots (fa_cache_evict): the positions below `first`
    and from next_pos[b] - last on are kept, then the slots of the largest weight (ties: the lowest slot);
    kept slots at or above `keep` move to the freed ones below.  weight [B, Hkv, capacity] float32 and
    pos int32 follow the slots, in place unless weight_out and pos_out are given.  Returns new_len [B]
    int32 = min(seq_len, keep); seq_len itself is not changed."""
    dev = cache.device
    slots = (cache.B, cache.Hkv, cache.capacity)
    if last and next_pos is None:
        raise ValueError("last needs next_pos")
    if new_len is None:
        new_len = torch.empty(cache.B, dtype=torch.int32, device=dev)
    w, p = _need("weight", weight, slots, torch.float32, dev), _need("pos", pos, slots, torch.int32, dev)
    args = (w, p, w if weight_out is None else _need("weight_out", weight_out, slots, torch.float32, dev),
            p if pos_out is None else _need("pos_out", pos_out, slots, torch.int32, dev),
            _need("new_len", new_len, (cache.B,), torch.int32, dev), _maybe("next_pos", next_pos, (cache.B,), torch.int32, dev))
    _check_stream_device(stream, dev)
    lib = _library()
    ws, size = _workspace(lib.fa_evict_workspace_bytes(cache.B, cache.Hkv, cache.capacity, keep), workspace, dev, stream)
    with _OnDevice(dev):
        _run(lib.fa_cache_evict(cache._ref, *args, keep, first, last, ws.data_ptr(), size, _stream_handle(stream)))
    return new_len
