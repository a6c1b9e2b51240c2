"""The cache operators' host side: the work schedule, the C ABI's refusals (made before any CUDA call)
and the binding's checks.  No GPU needed."""
import math
import os
import subprocess

import pytest
import torch

from programming_flashattention_fwd_gb300 import build as fa_build
from programming_flashattention_fwd_gb300 import cache as fc

HERE = os.path.dirname(os.path.abspath(__file__))


def test_schedule(tmp_path):
    """Every step to one CTA, equal shares, parts joined as they were cut (cache_schedule_check.cpp)."""
    exe = str(tmp_path / "cache_schedule_check")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(fa_build.nvcc()))), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{fa_build.CSRC}", f"-I{fa_build.INCLUDE}", f"-I{cuda}",
                    os.path.join(HERE, "cache_schedule_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fc._library()


# Fake, aligned, non-overlapping addresses: validation never dereferences them.
ADDR = {name: 0x1000000000 * (i + 1) for i, name in enumerate(
    ("k", "v", "table", "seq_len", "q", "k_new", "v_new", "parent", "draft_len", "o", "lse", "ws", "path", "count",
     "start", "weight", "pos", "weight_out", "pos_out", "new_len", "next_pos"))}
CACHE = dict(B=2, Hkv=2, D=128, page=64, max_pages=8, num_pages=20, dtype=0)


def cache_struct(**over):
    a = dict(CACHE, **{n: ADDR[n] for n in ("k", "v", "table", "seq_len")})
    a.update({k: v for k, v in over.items() if k in a})
    return fc._PACK(*(a[n] or 0 for n in ("k", "v", "table", "seq_len", "B", "Hkv", "D", "page", "max_pages", "num_pages", "dtype")))


def tree(lib, **over):
    a = dict(ADDR, Hq=4, T=5, scale=0.1, bytes=1 << 30)
    a.update(over)
    return lib.fa_tree_fwd(cache_struct(**over), a["q"], a["k_new"], a["v_new"], a["parent"], a["draft_len"], a["o"], a["lse"],
                           a["Hq"], a["T"], a["scale"], a["ws"], a["bytes"], None)


def append(lib, **over):
    a = dict(ADDR, T=5)
    a.update(over)
    return lib.fa_cache_append(cache_struct(**over), a["k_new"], a["v_new"], a["path"], a["count"], a["start"], a["weight"],
                               a["pos"], a["T"], None)


BAD_CACHE = [(dict(B=-1), 2), (dict(max_pages=-1), 2), (dict(num_pages=-1), 2), (dict(Hkv=0), 3), (dict(D=96), 4),
             (dict(D=32), 4), (dict(page=8), 2), (dict(page=24), 2), (dict(page=0), 2), (dict(dtype=2), 15),
             (dict(max_pages=1 << 26), 2), (dict(num_pages=0), 2), (dict(table=None, max_pages=11), 2), (dict(seq_len=None), 1),
             (dict(k=None), 1), (dict(v=None), 1), (dict(k=ADDR["k"] + 8), 5), (dict(seq_len=ADDR["seq_len"] + 2), 5)]


@pytest.mark.parametrize("over,code", BAD_CACHE + [
    (dict(Hq=3), 3), (dict(Hq=0), 3), (dict(T=-1), 2), (dict(scale=0.0), 7), (dict(scale=-0.1), 7), (dict(scale=math.nan), 7),
    (dict(scale=math.inf), 7), (dict(scale=3e38), 7), (dict(q=None), 1), (dict(k_new=None), 1), (dict(v_new=None), 1), (dict(o=None), 1),
    (dict(lse=None), 1), (dict(ws=None), 1), (dict(q=ADDR["q"] + 8), 5), (dict(lse=ADDR["lse"] + 2), 5),
    (dict(parent=ADDR["parent"] + 1), 5), (dict(ws=ADDR["ws"] + 16), 5), (dict(bytes=1000), 16), (dict(o=ADDR["q"]), 6),
    (dict(o=ADDR["k"] + 64), 6), (dict(lse=ADDR["o"] + 16), 6), (dict(ws=ADDR["v"]), 6), (dict(lse=ADDR["draft_len"]), 6),
    (dict(T=1 << 20, Hq=4096, Hkv=1, max_pages=100000), 2)])
def test_tree_refusals(lib, over, code):
    assert tree(lib, **over) == code


def test_tree_empty(lib):
    assert tree(lib, B=0, q=None, o=None, ws=None, bytes=0) == 0
    assert tree(lib, T=0, q=None, o=None, ws=None, bytes=0) == 0
    assert lib.fa_tree_workspace_bytes(4, 3, 1, 64) == 0 and lib.fa_tree_workspace_bytes(4, 2, 0, 64) == 0
    # the workspace depends on the rows of one KV head, up to one tile
    assert lib.fa_tree_workspace_bytes(8, 2, 1, 64) < lib.fa_tree_workspace_bytes(8, 2, 64, 64)
    assert lib.fa_tree_workspace_bytes(8, 2, 64, 64) == lib.fa_tree_workspace_bytes(8, 2, 640, 64)


@pytest.mark.parametrize("over,code", BAD_CACHE + [
    (dict(T=-1), 2), (dict(k_new=None), 1), (dict(v_new=None), 1), (dict(count=None), 1), (dict(start=None), 1),
    (dict(k_new=ADDR["k_new"] + 8), 5), (dict(path=ADDR["path"] + 2), 5), (dict(weight=ADDR["weight"] + 1), 5),
    (dict(k_new=ADDR["k"]), 6), (dict(weight=ADDR["pos"]), 6), (dict(pos=ADDR["seq_len"]), 6), (dict(v=ADDR["k"]), 6)])
def test_append_refusals(lib, over, code):
    assert append(lib, **over) == code


def test_append_empty(lib):
    assert append(lib, B=0, k_new=None) == 0 and append(lib, T=0, k_new=None) == 0


def weights(lib, **over):
    a = dict(ADDR, Hq=4, T=5, causal=1, scale=0.1, bytes=1 << 30)
    a.update(over)
    return lib.fa_cache_weights(cache_struct(**over), a["q"], a["lse"], a["path"], a["count"], a["weight"], a["weight_out"], a["Hq"],
                                a["T"], a["causal"], a["scale"], a["ws"], a["bytes"], None)


def evict(lib, **over):
    a = dict(ADDR, keep=100, first=4, last=16, bytes=1 << 30)
    a.update(over)
    return lib.fa_cache_evict(cache_struct(**over), a["weight"], a["pos"], a["weight_out"], a["pos_out"], a["new_len"], a["next_pos"],
                              a["keep"], a["first"], a["last"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("over,code", BAD_CACHE + [
    (dict(Hq=3), 3), (dict(Hq=0), 3), (dict(T=-1), 2), (dict(T=0), 2), (dict(scale=0.0), 7), (dict(scale=math.nan), 7),
    (dict(causal=2), 13), (dict(causal=-1), 13), (dict(q=None), 1), (dict(lse=None), 1), (dict(count=None), 1),
    (dict(weight_out=None), 1), (dict(ws=None), 1), (dict(q=ADDR["q"] + 8), 5), (dict(lse=ADDR["lse"] + 2), 5),
    (dict(weight=ADDR["weight"] + 1), 5), (dict(ws=ADDR["ws"] + 4), 5), (dict(bytes=100), 16), (dict(weight_out=ADDR["weight"] + 4), 6),
    (dict(weight_out=ADDR["k"]), 6), (dict(ws=ADDR["lse"]), 6), (dict(weight_out=ADDR["seq_len"]), 6),
    (dict(B=1, Hkv=1, Hq=64, T=1 << 20, max_pages=1 << 16, num_pages=1 << 16), 2)])
def test_weights_refusals(lib, over, code):
    assert weights(lib, **over) == code


@pytest.mark.parametrize("over,code", BAD_CACHE + [
    (dict(keep=0), 2), (dict(first=-1), 2), (dict(last=-1), 2), (dict(first=50, last=51), 2), (dict(weight=None), 1), (dict(pos=None), 1),
    (dict(weight_out=None), 1), (dict(pos_out=None), 1), (dict(new_len=None), 1), (dict(next_pos=None), 1), (dict(ws=None), 1),
    (dict(bytes=1000), 16), (dict(weight=ADDR["weight"] + 2), 5), (dict(new_len=ADDR["new_len"] + 1), 5), (dict(ws=ADDR["ws"] + 2), 5),
    (dict(weight_out=ADDR["weight"] + 4), 6), (dict(pos_out=ADDR["weight"]), 6), (dict(new_len=ADDR["seq_len"]), 6),
    (dict(new_len=ADDR["next_pos"]), 6), (dict(ws=ADDR["pos"]), 6), (dict(weight_out=ADDR["v"]), 6), (dict(k=ADDR["v"]), 6)])
def test_evict_refusals(lib, over, code):
    assert evict(lib, **over) == code


def test_weights_and_evict_empty(lib):
    assert weights(lib, B=0, q=None) == 0 and weights(lib, max_pages=0, q=None) == 0
    assert evict(lib, B=0, weight=None) == 0
    assert lib.fa_evict_workspace_bytes(2, 2, 100, 100) == 0 and lib.fa_evict_workspace_bytes(2, 2, 100, 90) == 2 * 2 * 10 * 16


class FakeCuda(torch.Tensor):
    """A CPU tensor that reports itself as living on a given CUDA device (no GPU needed)."""
    _dev = torch.device("cuda", 0)

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return self._dev

    def get_device(self):
        return self._dev.index


def on(shape, dtype=torch.bfloat16, idx=0):
    t = torch.Tensor._make_subclass(FakeCuda, torch.zeros(shape, dtype=dtype))
    t._dev = torch.device("cuda", idx)
    return t


def make_cache(**over):
    a = dict(k=on((6, 2, 16, 64)), v=on((6, 2, 16, 64)), seq_len=on((2,), torch.int32), table=on((2, 3), torch.int32))
    a.update(over)
    return fc.KVCache(**a)


@pytest.mark.parametrize("over,what", [
    (dict(k=torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)), "CUDA"), (dict(k=on((6, 2, 16, 64), torch.float32)), "bf16 or fp16"),
    (dict(v=on((6, 2, 16, 64), torch.float16)), "v must be"), (dict(v=on((6, 2, 8, 64))), "shape"),
    (dict(v=on((6, 2, 16, 64), idx=1)), "same GPU"), (dict(seq_len=on((2,), torch.int64)), "seq_len"),
    (dict(table=on((3, 3), torch.int32)), "table"), (dict(table=on((3,), torch.int32)), "table"), (dict(k=on((6, 2, 16))), "k must be")])
def test_cache_checks_its_tensors(over, what):
    with pytest.raises(ValueError, match=what):
        make_cache(**over)


def test_dense_cache_shares_its_pages_out():
    assert make_cache(table=None).capacity == 48 and make_cache().capacity == 48
    assert make_cache(table=None, seq_len=on((4,), torch.int32)).capacity == 16


def tree_args(**over):
    a = dict(q=on((2, 4, 5, 64)), k_new=on((2, 2, 5, 64)), v_new=on((2, 2, 5, 64)), cache=make_cache(), parent=on((2, 5), torch.int32),
             draft_len=on((2,), torch.int32), o=on((2, 4, 5, 64)), lse=on((2, 4, 5), torch.float32))
    a.update(over)
    return a


@pytest.mark.parametrize("over,what", [
    (dict(q=on((3, 4, 5, 64))), "sequences"), (dict(q=on((2, 4, 5, 128))), "head dimension"), (dict(q=on((2, 4, 5, 64), torch.float16)), "q must be"),
    (dict(k_new=on((2, 4, 5, 64))), "k_new"), (dict(parent=on((2, 4), torch.int32)), "parent"), (dict(draft_len=on((2,), torch.int64)), "draft_len"),
    (dict(o=on((2, 4, 5, 64), idx=1)), "same GPU"), (dict(lse=on((2, 4, 5))), "lse"),
    (dict(q=on((2, 5, 4, 64)).transpose(1, 2)), "contiguous")])
def test_tree_attention_checks_its_tensors(over, what, monkeypatch, lib):
    called = []
    monkeypatch.setattr(fc, "_launch", lambda *a: called.append(1))
    with pytest.raises(ValueError, match=what):
        fc.tree_attention(**tree_args(**over))
    assert not called


@pytest.mark.parametrize("over,what", [
    (dict(k_new=on((2, 3, 5, 64))), "k_new"), (dict(path=on((2, 5), torch.int32)), "needs count"),
    (dict(pos=on((2, 2, 48), torch.int32)), "needs start"), (dict(weight=on((2, 2, 40), torch.float32)), "weight"),
    (dict(count=on((3,), torch.int32)), "count")])
def test_cache_append_checks_its_tensors(over, what):
    a = dict(cache=make_cache(), k_new=on((2, 2, 5, 64)), v_new=on((2, 2, 5, 64)))
    a.update(over)
    with pytest.raises(ValueError, match=what):
        fc.cache_append(**a)


@pytest.mark.parametrize("over,what", [
    (dict(q=on((2, 4, 5, 128))), "head dimension"), (dict(lse=on((2, 4, 6), torch.float32)), "lse"), (dict(path=on((2, 5), torch.int32)), "needs count"),
    (dict(weight=on((2, 2, 48))), "weight"), (dict(out=on((2, 2, 49), torch.float32)), "out"), (dict(lse=on((2, 4, 5), torch.float32, 1)), "same GPU")])
def test_cache_weights_checks_its_tensors(over, what):
    a = dict(cache=make_cache(), q=on((2, 4, 5, 64)), lse=on((2, 4, 5), torch.float32), weight=on((2, 2, 48), torch.float32))
    a.update(over)
    with pytest.raises(ValueError, match=what):
        fc.cache_weights(**a)


@pytest.mark.parametrize("over,what", [
    (dict(last=3), "needs next_pos"), (dict(keep=0), "positive"), (dict(keep=2 ** 32 + 5), "positive"), (dict(first=-1), "negative"), (dict(weight=on((2, 2, 40), torch.float32)), "weight"), (dict(pos=on((2, 2, 48), torch.int64)), "pos"),
    (dict(pos_out=on((2, 2, 48), torch.float32)), "pos_out"), (dict(new_len=on((3,), torch.int32)), "new_len"),
    (dict(next_pos=on((2,), torch.int32, 1)), "same GPU")])
def test_cache_evict_checks_its_tensors(over, what):
    a = dict(cache=make_cache(), weight=on((2, 2, 48), torch.float32), pos=on((2, 2, 48), torch.int32), keep=20, new_len=on((2,), torch.int32))
    a.update(over)
    with pytest.raises(ValueError, match=what):
        fc.cache_evict(**a)


def test_struct_is_the_header_s(tmp_path):
    """The packed fields of the binding against the C compiler's layout of fa_cache_t."""
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fa.h"\nint main(void) { printf("%zu %zu %zu %zu %zu\\n", sizeof(fa_cache_t), '
                   'offsetof(fa_cache_t, seq_len), offsetof(fa_cache_t, B), offsetof(fa_cache_t, page), offsetof(fa_cache_t, dtype)); return 0; }\n')
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", f"-I{fa_build.INCLUDE}", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    packed = fc._PACK(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11)
    assert got == [len(packed), 24, 32, 44, 56]
    assert packed[32:60] == b"".join(x.to_bytes(4, "little") for x in range(5, 12))
