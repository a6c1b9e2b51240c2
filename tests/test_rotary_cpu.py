"""Rotary operators without a GPU: the calls that they refuse, the layout of what the binding passes, the frequencies."""
import ctypes
import math
import struct

import pytest

from programming_flashattention_fwd_gb300 import build as fa_build


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    from programming_flashattention_fwd_gb300 import positions
    return positions._library()


class Table(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("D", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("amplitude", ctypes.c_float)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64), ("stride_t", ctypes.c_int64), ("heads", ctypes.c_int)]


def test_structs_as_the_binding_packs_them():
    from programming_flashattention_fwd_gb300 import positions as m
    assert bytes(Table(1 << 40, 128, 64, 1, 0.5)) == m._TABLE(1 << 40, 128, 64, 1, 0.5)
    assert bytes(Heads(1 << 40, 5, 6, 7, 8))[:36] == m._HEADS(1 << 40, 5, 6, 7, 8)[:36] and len(m._HEADS(0, 0, 0, 0, 0)) == ctypes.sizeof(Heads)


# Addresses that validation never reads.
F, Q, K, QO, KO, ST, PO = ((i + 1) << 40 for i in range(7))
B, T, D, HQ, HK = 2, 50, 64, 4, 2


def heads(at, n, sb=None, sh=None, st=None):
    return Heads(at, n * T * D if sb is None else sb, T * D if sh is None else sh, D if st is None else st, n)


def call(lib, table=None, x=None, y=None, n=2, B=B, T=T, start=ST, position=None, inverse=0, dtype=0):
    table = Table(F, D, D, 0, 1.0) if table is None else table
    x = (Heads * 2)(*(x or (heads(Q, HQ), heads(K, HK))))
    y = (Heads * 2)(*(y or (heads(QO, HQ), heads(KO, HK))))
    return lib.fa_rotary(bytes(table), bytes(x), bytes(y), n, B, T, start, position, inverse, dtype, None)


def row(at, n, width, off):
    """n heads from element `off` of rows of `width` elements."""
    return heads(at + 2 * off, n, T * width, D, width)


@pytest.mark.parametrize("over,code", [
    (dict(table=Table(F, 96, 32, 0, 1.0)), 4), (dict(table=Table(F, D, 7, 0, 1.0)), 2), (dict(table=Table(F, D, 66, 0, 1.0)), 2),
    (dict(table=Table(F, D, -2, 0, 1.0)), 2), (dict(table=Table(F, D, D, 2, 1.0)), 15), (dict(table=Table(F, D, D, 0, math.inf)), 7),
    (dict(table=Table(F, D, D, 0, math.nan)), 7), (dict(table=Table(None, D, D, 0, 1.0)), 1), (dict(table=Table(F + 4, D, D, 0, 1.0)), 5),
    (dict(n=0), 15), (dict(n=3), 15), (dict(inverse=2), 15), (dict(dtype=2), 15), (dict(position=PO), 15), (dict(B=-1), 2), (dict(T=-1), 2),
    (dict(T=2 ** 31 - 1, B=2 ** 31 - 1), 2), (dict(start=ST + 2), 5), (dict(start=None, position=PO + 2), 5),
    (dict(x=(heads(None, HQ), heads(K, HK))), 1), (dict(y=(heads(QO, HQ), heads(None, HK))), 1), (dict(x=(heads(Q, HQ), heads(K, -1))), 3),
    (dict(y=(heads(QO, HQ + 1), heads(KO, HK))), 3), (dict(x=(heads(Q, 70000), heads(K, HK)), y=(heads(QO, 70000), heads(KO, HK))), 2),
    (dict(x=(heads(Q + 8, HQ), heads(K, HK))), 5), (dict(y=(heads(QO, HQ, st=D + 4), heads(KO, HK))), 5),
    (dict(x=(heads(Q, HQ, sh=-T * D), heads(K, HK))), 2),
    # a result whose heads or tokens share a place; one over an input, over the other, over the positions
    (dict(y=(heads(QO, HQ, sh=0), heads(KO, HK))), 6), (dict(y=(heads(QO, HQ, st=D - 8), heads(KO, HK))), 6), (dict(y=(heads(QO, HQ, sb=0), heads(KO, HK))), 6),
    (dict(y=(heads(K, HQ), heads(KO, HK))), 6), (dict(y=(heads(QO, HQ), heads(QO, HK))), 6), (dict(y=(heads(Q + 16, HQ), heads(KO, HK))), 6),
    (dict(y=(heads(Q, HQ, sb=HQ * T * D + 8), heads(KO, HK))), 6), (dict(y=(heads(ST, HQ), heads(KO, HK))), 6), (dict(y=(heads(F, HQ), heads(KO, HK))), 6),
    # heads of one projection's rows that overlap by 8 elements, or reach into the next row
    (dict(y=(row(QO, HQ, 512, 0), row(QO, HK, 512, HQ * D - 8))), 6), (dict(y=(row(QO, HQ, 376, 0), row(QO, HK, 376, HQ * D))), 6),
])
def test_refusals(lib, over, code):
    assert call(lib, **over) == code


def test_nothing_to_do(lib):
    assert call(lib, B=0) == 0 and call(lib, T=0) == 0
    assert call(lib, x=(heads(None, 0), heads(None, 0)), y=(heads(None, 0), heads(None, 0))) == 0


def test_heads_side_by_side_pass_the_checks(lib):
    """Views of the rows of one projection are not refused; the call stops at the missing device, or, where there is one,
    is not made."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would run on made-up addresses")
    assert call(lib, x=(row(Q, HQ, 512, 0), row(Q, HK, 512, HQ * D)), y=(row(QO, HQ, 512, 0), row(QO, HK, 512, HQ * D))) == 8
    assert call(lib, x=(row(Q, HQ, 384, 0), row(Q, HK, 384, HQ * D)), y=(row(Q, HQ, 384, 0), row(Q, HK, 384, HQ * D))) == 8   # in place
    assert call(lib, x=(heads(Q, HQ, sh=0), heads(K, HK))) == 8   # one head read several times
    whole = (HQ + HK) * T * D   # heads of one dense tensor
    assert call(lib, y=(heads(QO, HQ, sb=whole), heads(QO + 2 * HQ * T * D, HK, sb=whole))) == 8
    assert call(lib, y=(heads(QO, HQ, sb=whole), heads(QO + 2 * (HQ - 1) * T * D, HK, sb=whole))) == 6
    assert call(lib, y=(heads(QO, HQ, sb=whole), heads(QO + 2 * (HQ + 1) * T * D, HK, sb=whole))) == 6   # into the next sequence


def test_rows_that_interleave_are_refused(lib):
    """Two views whose rows are apart from token to token, but whose sequences begin between each other's tokens."""
    wx, wy = HQ * D, HK * D
    rows = lambda at, n, off: heads(at + 2 * off, n, wy + wx + wy, D, wx + wy)  # noqa: E731
    assert call(lib, T=2, y=(rows(QO, HQ, 0), rows(QO, HK, wx))) == 6
    assert call(lib, T=2, x=(rows(QO, HQ, 0), heads(K, HK)), y=(heads(KO, HQ), rows(QO, HK, wx))) == 6
    far = 2 ** 60   # the ends of such views do not fit 64 bits
    assert call(lib, x=(heads(Q, HQ, far, far, far), heads(K, HK))) == 2


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "table", "seq_len")] + [(n, ctypes.c_int) for n in ("B", "Hkv", "D", "page", "max_pages", "num_pages", "dtype")]


KP, VP, TB, SL, V, VO, CN, WT, PS = ((i + 20) << 40 for i in range(9))
CACHE = dict(k=KP, v=VP, table=TB, seq_len=SL, B=B, Hkv=HK, D=D, page=16, max_pages=8, num_pages=20, dtype=0)


def append(lib, cache=(), table=None, x=None, y=None, T=T, start=ST, position=None, count=CN, weight=WT, pos=PS):
    c = Cache(*(dict(CACHE, **dict(cache))[n] for n, _ in Cache._fields_))
    x = (Heads * 3)(*(x or (heads(Q, HQ), heads(K, HK), heads(V, HK))))
    y = (Heads * 3)(*(y or (heads(QO, HQ), heads(KO, HK), heads(VO, HK))))
    return lib.fa_rotary_append(bytes(c), bytes(table or Table(F, D, D, 0, 1.0)), bytes(x), bytes(y), T, start, position, count, weight, pos, None)


@pytest.mark.parametrize("over,code", [
    (dict(cache=dict(page=8)), 2), (dict(cache=dict(D=128)), 4), (dict(cache=dict(dtype=2)), 15), (dict(cache=dict(seq_len=None)), 1), (dict(cache=dict(k=KP + 8)), 5),
    (dict(position=PO), 15), (dict(T=-1), 2), (dict(x=(heads(Q, 3), heads(K, HK), heads(V, HK)), y=(heads(QO, 3), heads(KO, HK), heads(VO, HK))), 3),
    (dict(x=(heads(Q, HQ), heads(K, 1), heads(V, HK)), y=(heads(QO, HQ), heads(KO, 1), heads(VO, HK))), 3),
    (dict(x=(heads(Q, HQ), heads(None, HK), heads(V, HK))), 1), (dict(count=CN + 2), 5), (dict(weight=WT + 2), 5), (dict(pos=PS + 1), 5),
    (dict(y=(heads(QO, HQ), heads(KP, HK), heads(VO, HK))), 6), (dict(x=(heads(Q, HQ), heads(K, HK), heads(VP + 64, HK))), 6), (dict(weight=PS), 6),
    (dict(weight=KP + 64), 6), (dict(pos=SL), 6), (dict(y=(heads(QO, HQ), heads(CN, HK), heads(VO, HK))), 6), (dict(y=(heads(QO, HQ), heads(TB, HK), heads(VO, HK))), 6),
    (dict(pos=F), 6), (dict(cache=dict(k=ST)), 6),
])
def test_append_refusals(lib, over, code):
    assert append(lib, **over) == code


def test_append_nothing_to_do(lib):
    assert append(lib, T=0) == 0 and append(lib, cache=dict(B=0)) == 0


def test_frequencies():
    import programming_flashattention_fwd_gb300 as fa
    f = fa.rotary_frequencies(64)
    assert len(f) == 32 and f[0] == 1.0 and abs(f[-1] - 10000.0 ** (-62 / 64)) < 1e-18
    assert fa.rotary_frequencies(64, scaling="linear", factor=4.0) == [x / 4 for x in f]
    b = fa.rotary_frequencies(64, scaling="base", factor=8.0)
    assert b[0] == 1.0 and abs(b[-1] - f[-1] / 8) < 1e-15
    r = fa.rotary_frequencies(128, scaling="ramp", factor=8.0, original=4096)
    f = fa.rotary_frequencies(128)
    turns = [4096 * x / (2 * math.pi) for x in f]
    assert all(x == y for x, y, t in zip(r, f, turns) if t > 40) and all(abs(x - y / 8) < 1e-18 for x, y, t in zip(r, f, turns) if t < 0.8)
    assert all(y / 8 <= x * (1 + 1e-12) and x <= y for x, y in zip(r, f)) and all(x > y for x, y in zip(r, r[1:]))
    for bad in (dict(rot=7), dict(rot=64, scaling="other"), dict(rot=64, scaling="ramp", factor=2.0), dict(rot=2, scaling="base", factor=2.0), dict(rot=64, base=0.0)):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(**bad)


def test_table_struct_holds_the_packed_cache():
    assert ctypes.sizeof(Cache) == struct.calcsize("PPPP7i4x") and ctypes.sizeof(Table) == 24
