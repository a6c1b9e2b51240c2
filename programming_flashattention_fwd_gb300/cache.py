"""Operators of a paged key/value cache: argument marshalling over libfa_gb300.so.

``KVCache`` names the tensors of one layer's cache; ``tree_attention`` attends drafted tokens over
it, ``cache_append`` writes accepted tokens, ``cache_weights`` adds up the attention that each slot
receives and ``cache_evict`` shrinks the cache by it.  include/fa.h defines each operator; as in
``binding``, every step of the computation runs in the library's CUDA kernels and a non-zero
status raises ``FaError``.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import struct
import threading
from typing import Optional, Tuple

import torch

from . import binding as _b
from .binding import FaError, _check_stream_device, _OnDevice, _stream_handle, fa_strerror, load_library

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_I32, _F32 = torch.int32, torch.float32

# fa_cache_t of include/fa.h: k, v, table, seq_len; B, Hkv, D, page, max_pages, num_pages, dtype
_PACK = struct.Struct("PPPP7i4x").pack

_P, _I, _F, _Z, _C = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_char_p
_SIGNATURES = {
    "fa_tree_workspace_bytes": (_Z, [_I] * 4),
    "fa_tree_fwd": (_I, [_C] + [_P] * 7 + [_I, _I, _F, _P, _Z, _P]),
    "fa_cache_append": (_I, [_C] + [_P] * 7 + [_I, _P]),
    "fa_weights_workspace_bytes": (_Z, []),
    "fa_cache_weights": (_I, [_C] + [_P] * 6 + [_I, _I, _I, _F, _P, _Z, _P]),
    "fa_tree_debug": (_I, [_C] + [_P] * 7 + [_I, _I, _F, _P, _Z, _P, ctypes.c_uint64, ctypes.c_uint32]),
    "fa_weights_debug": (_I, [_C] + [_P] * 6 + [_I, _I, _I, _F, _P, _Z, _P, ctypes.c_uint64, ctypes.c_uint32]),
    "fa_evict_workspace_bytes": (_Z, [_I] * 4),
    "fa_cache_evict": (_I, [_C] + [_P] * 6 + [_I, _I, _I, _P, _Z, _P]),
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


def _refuse(name: str, t, shape, dtype, index: int):
    """What is wrong with a tensor that _need does not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device} but the cache is on cuda:{index}: "
                         "every tensor of one call must be on the same GPU")
    raise ValueError(f"{name} must be contiguous")


def _need(name: str, t, shape, dtype, index: int) -> int:
    """The address of a dense CUDA tensor of this shape and type on this device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(name, t, shape, dtype, index)


def _on(stream, cache: "KVCache", fn, *args):
    """fn(*args) with `stream` (a torch.cuda.Stream or a handle) current.  What the call allocates and fills then
    belongs to that stream: memory of the current stream's may still be in use by what runs there."""
    device = cache.device
    _check_stream_device(stream, device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    user = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        result = fn(*args)
    # results are for the caller's stream, which may outlast their last reference
    for t in result if isinstance(result, tuple) else (result,):
        if t is not None:
            t.record_stream(user)
    return result


def _current(index: int) -> Optional[int]:
    """The handle of the current stream, if the cache's device is the current one."""
    if _b._raw_stream is not None and _b._cur_device is not None and _b._cur_device() == index:
        return _b._raw_stream(index)
    return None


def _launch(fn, index: int, current: Optional[int], args) -> None:
    """fn(*args, stream handle) with the cache's device current; raises on a non-zero status."""
    if current is not None:
        st = fn(*args, current)
    else:
        with _OnDevice(torch.device("cuda", index)):
            st = fn(*args, _stream_handle(None))
    if st != 0:
        raise FaError(st, fa_strerror(st))


_local = threading.local()
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _kept(index: int, current: Optional[int]) -> Optional[dict]:
    """What this thread keeps for the current stream, whose calls run one after another: its workspace.  None
    where a call is to have its own: on another device than the current one, or captured into a graph."""
    if current is None or _capturing():
        return None
    kept, key = _local.__dict__, (index, current)
    entry = kept.get(key)
    if entry is None:
        entry = kept[key] = {}
    return entry


def _workspace(need: int, given: Optional[torch.Tensor], like: torch.Tensor, kept) -> Tuple[torch.Tensor, int, int]:
    """A workspace on like's device, its address and size: the caller's, the kept one, or one for this call."""
    if given is not None:
        if given.get_device() != like.get_device() or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the cache's device")
        return given, given.data_ptr(), given.nbytes
    if kept is not None:
        ws = kept.get("workspace")
        if ws is None or ws[2] < need:
            t = torch.empty(need, dtype=torch.uint8, device=like.device)
            ws = kept["workspace"] = (t, t.data_ptr(), need)
        return ws
    t = torch.empty(need, dtype=torch.uint8, device=like.device)
    return t, t.data_ptr(), need


def _fixed(name: str) -> property:
    """A tensor of a KVCache, whose address the cache's calls pass on: another one in its place would not be seen by
    them, so only the same one may be assigned (which is what `cache.seq_len += count` does after it has added)."""
    def assign(self, t):
        if t is not getattr(self, "_" + name):
            raise AttributeError(f"a KVCache keeps the {name} that it was made with: change that in place, or make another KVCache")
    return property(operator.attrgetter("_" + name), assign)


class KVCache:
    """The keys and values of B sequences in pages (fa_cache_t).

    k, v     [num_pages, Hkv, page, D] bf16 or fp16, contiguous CUDA tensors; page a multiple of 16
    seq_len  [B] int32: slots in use of each sequence, read by the kernels when they run
    table    [B, max_pages] int32: the page of each run of `page` slots; None for a dense cache,
             whose pages belong to the sequences in order (num_pages // B each)

    Holds references to the tensors and no state of its own: update seq_len and table in place (another tensor in
    their place is refused).
    """
    __slots__ = ("_k", "_v", "_seq_len", "_table", "index", "dtype", "B", "Hkv", "D", "page", "capacity", "_c")
    k, v, seq_len, table = (_fixed(name) for name in ("k", "v", "seq_len", "table"))

    def __init__(self, k: torch.Tensor, v: torch.Tensor, seq_len: torch.Tensor, table: Optional[torch.Tensor] = None):
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a [num_pages, Hkv, page, D] tensor")
        code = _DTYPES.get(k.dtype)
        if code is None:
            raise ValueError(f"a cache is bf16 or fp16, not {k.dtype}")
        index = k.get_device()
        if index < 0:
            raise ValueError("k must be a CUDA tensor")
        shape = k.shape
        num, Hkv, page, D = shape
        if not isinstance(seq_len, torch.Tensor) or seq_len.dim() != 1:
            raise ValueError("seq_len must be a [B] tensor")
        B = seq_len.shape[0]
        if table is None:
            per, at = num // B if B else 0, 0
        else:
            if not isinstance(table, torch.Tensor) or table.dim() != 2:
                raise ValueError("table must be a [B, max_pages] tensor")
            per = table.shape[1]
            at = _need("table", table, (B, per), _I32, index)
        dt = k.dtype
        if not k.is_contiguous():
            raise ValueError("k must be contiguous")
        self._c = _PACK(k.data_ptr(), _need("v", v, shape, dt, index), at,
                        _need("seq_len", seq_len, (B,), _I32, index), B, Hkv, D, page, per, num, code)
        self._k, self._v, self._seq_len, self._table = k, v, seq_len, table
        self.index, self.dtype, self.B, self.Hkv, self.D, self.page = index, dt, B, Hkv, D, page
        self.capacity = per * page

    @property
    def device(self) -> torch.device:
        return self._k.device

    def __reduce__(self):
        # a copy is made from its tensors: a deep one has others, at other addresses
        return KVCache, (self._k, self._v, self._seq_len, self._table)


@functools.lru_cache(maxsize=256)
def tree_workspace_bytes(Hq: int, Hkv: int, T: int, D: int) -> int:
    """Bytes of the workspace of ``tree_attention`` for T drafted tokens."""
    return _library().fa_tree_workspace_bytes(Hq, Hkv, T, D)


def _queries(q, cache: KVCache):
    """The sizes of q [B, Hq, T, D], which must fit the cache."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, Hq, T, D] tensor")
    shape = q.shape
    if shape[0] != cache.B or shape[3] != cache.D:
        raise ValueError(f"q must have the cache's {cache.B} sequences and head dimension {cache.D}")
    return shape


def tree_attention(q, k_new, v_new, cache: KVCache, parent=None, draft_len=None, scale: Optional[float] = None,
                   o=None, lse=None, workspace=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of drafted tokens over the cache and over the drafted tokens on their path (fa_tree_fwd).

    q [B, Hq, T, D], k_new and v_new [B, Hkv, T, D] in the cache's type; parent [B, T] int32 (-1: a
    root; None: a chain), draft_len [B] int32 (None: T).  Returns (o [B, Hq, T, D], lse [B, Hq, T]
    float32), in o and lse where they are given; rows at or behind draft_len are not written.
    scale defaults to D ** -0.5.  workspace: tree_workspace_bytes(...) bytes that no other call in
    flight uses; None: one that is kept for the calling thread and the stream, or, in a call that is
    captured into a graph, one of the graph's own.  stream (of this and the other operators): where the call
    runs, and what it allocates then belongs to; None: the current stream."""
    if stream is not None:
        return _on(stream, cache, tree_attention, q, k_new, v_new, cache, parent, draft_len, scale, o, lse, workspace)
    shape = _queries(q, cache)
    B, Hq, T, D = shape
    i, dt, Hkv = cache.index, cache.dtype, cache.Hkv
    new, rows = (B, Hkv, T, D), (B, Hq, T)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(rows, dtype=_F32, device=q.device)
    lib = _lib or _library()
    args = (cache._c, _need("q", q, shape, dt, i), _need("k_new", k_new, new, dt, i), _need("v_new", v_new, new, dt, i),
            None if parent is None else _need("parent", parent, (B, T), _I32, i),
            None if draft_len is None else _need("draft_len", draft_len, (B,), _I32, i),
            _need("o", o, shape, dt, i), _need("lse", lse, rows, _F32, i), Hq, T, D ** -0.5 if scale is None else scale)
    current = _current(i)
    ws, at, size = _workspace(tree_workspace_bytes(Hq, Hkv, T, D), workspace, q, _kept(i, current))
    _launch(lib.fa_tree_fwd, i, current, args + (at, size))
    return o, lse


def cache_append(cache: KVCache, k_new, v_new, path=None, count=None, weight=None, pos=None, start=None,
                 stream=None) -> None:
    """Writes tokens behind the slots in use (fa_cache_append): slot seq_len[b] + i takes token path[b, i]
    (token i without a path) of k_new, v_new [B, Hkv, T, D], i < count[b] (None: T).  weight
    [B, Hkv, capacity] float32 becomes 0 and pos [B, Hkv, capacity] int32 start[b] + i at the new slots,
    where given.  seq_len is not changed: add count to it after the last layer."""
    if stream is not None:
        return _on(stream, cache, cache_append, cache, k_new, v_new, path, count, weight, pos, start)
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4:
        raise ValueError("k_new must be a [B, Hkv, T, D] tensor")
    i, dt, B, Hkv, T = cache.index, cache.dtype, cache.B, cache.Hkv, k_new.shape[2]
    new, slots = (B, Hkv, T, cache.D), (B, Hkv, cache.capacity)
    if path is not None and count is None:
        raise ValueError("a path needs count")
    if pos is not None and start is None:
        raise ValueError("pos needs start")
    lib = _lib or _library()
    args = (cache._c, _need("k_new", k_new, new, dt, i), _need("v_new", v_new, new, dt, i),
            None if path is None else _need("path", path, (B, T), _I32, i),
            None if count is None else _need("count", count, (B,), _I32, i),
            None if start is None else _need("start", start, (B,), _I32, i),
            None if weight is None else _need("weight", weight, slots, _F32, i),
            None if pos is None else _need("pos", pos, slots, _I32, i), T)
    _launch(lib.fa_cache_append, i, _current(i), args)


@functools.lru_cache(maxsize=1)
def weights_workspace_bytes() -> int:
    """Bytes of the workspace of ``cache_weights``."""
    return _library().fa_weights_workspace_bytes()


def cache_weights(cache: KVCache, q, lse, weight=None, path=None, count=None, causal: bool = True,
                  scale: Optional[float] = None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Adds to each slot the attention weight that it receives from the rows of q (fa_cache_weights).

    q [B, Hq, T, D], lse [B, Hq, T] as the attention left it; path [B, T] and count [B] int32 as in
    ``cache_append`` (the accepted rows); causal: row i is the query of slot seq_len[b] - count[b] + i
    and sees the slots up to its own.  weight [B, Hkv, capacity] float32 (None: zeros) is added to; the
    result is written to out, which defaults to weight itself (without a weight, to a new tensor of zeros).  For
    accepted tokens it follows their append in every layer and seq_len += count."""
    if stream is not None:
        return _on(stream, cache, cache_weights, cache, q, lse, weight, path, count, causal, scale, out, workspace)
    shape = _queries(q, cache)
    B, Hq, T, D = shape
    i = cache.index
    if path is not None and count is None:
        raise ValueError("a path needs count")
    slots = (B, cache.Hkv, cache.capacity)
    if out is None:
        out = torch.zeros(slots, dtype=_F32, device=q.device) if weight is None else weight
    lib = _lib or _library()
    args = (cache._c, _need("q", q, shape, cache.dtype, i), _need("lse", lse, (B, Hq, T), _F32, i),
            None if path is None else _need("path", path, (B, T), _I32, i),
            None if count is None else _need("count", count, (B,), _I32, i),
            None if weight is None else _need("weight", weight, slots, _F32, i), _need("out", out, slots, _F32, i),
            Hq, T, 1 if causal else 0, D ** -0.5 if scale is None else scale)
    current = _current(i)
    ws, at, size = _workspace(weights_workspace_bytes(), workspace, q, _kept(i, current))
    _launch(lib.fa_cache_weights, i, current, args + (at, size))
    return out


@functools.lru_cache(maxsize=256)
def evict_workspace_bytes(B: int, Hkv: int, capacity: int, keep: int) -> int:
    """Bytes of the workspace of ``cache_evict``."""
    return _library().fa_evict_workspace_bytes(B, Hkv, capacity, keep)


def cache_evict(cache: KVCache, weight, pos, keep: int, first: int = 0, last: int = 0, next_pos=None, weight_out=None,
                pos_out=None, new_len=None, workspace=None, stream=None) -> torch.Tensor:
    """Shrinks every sequence and KV head to `keep` slots (fa_cache_evict): the positions below `first`
    and from next_pos[b] - last on are kept, then the slots of the largest weight (ties: the lowest slot);
    kept slots at or above `keep` move to the freed ones below.  weight [B, Hkv, capacity] float32 and
    pos int32 follow the slots, in place unless weight_out and pos_out are given.  Returns new_len [B]
    int32 = min(seq_len, keep), a tensor of its own unless one is given (which saves the host an allocation);
    seq_len itself is not changed: the layers of a model share it, and one that found it shortened would evict
    nothing and lose the slots behind.  Copy new_len into it after the last layer."""
    if stream is not None:
        return _on(stream, cache, cache_evict, cache, weight, pos, keep, first, last, next_pos, weight_out, pos_out, new_len,
                   workspace)
    i, B = cache.index, cache.B
    slots = (B, cache.Hkv, cache.capacity)
    if last and next_pos is None:
        raise ValueError("last needs next_pos")
    if not 0 < keep < 2 ** 31 or not 0 <= first < 2 ** 31 or not 0 <= last < 2 ** 31:
        raise ValueError("keep must be positive, first and last not negative")
    w, p = _need("weight", weight, slots, _F32, i), _need("pos", pos, slots, _I32, i)
    wo = w if weight_out is None else _need("weight_out", weight_out, slots, _F32, i)
    po = p if pos_out is None else _need("pos_out", pos_out, slots, _I32, i)
    nxt = None if next_pos is None else _need("next_pos", next_pos, (B,), _I32, i)
    if new_len is not None:
        _need("new_len", new_len, (B,), _I32, i)
    lib = _lib or _library()
    current = _current(i)
    kept = _kept(i, current)
    if new_len is None:
        new_len = torch.empty_like(cache.seq_len)
    ws, at, size = _workspace(evict_workspace_bytes(B, cache.Hkv, cache.capacity, keep), workspace, cache.k, kept)
    _launch(lib.fa_cache_evict, i, current,
            (cache._c, w, p, wo, po, new_len.data_ptr(), nxt, keep, first, last, at, size))
    return new_len
