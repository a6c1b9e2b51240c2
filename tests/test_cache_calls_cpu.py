"""Calls of the cache operators as a user's program makes them, as far as they go without a GPU: what a call returns
and what it does with the tensors that it is given."""
import copy
import io
import os
import re

import pytest
import torch

from programming_flashattention_fwd_gb300 import build as fa_build
from programming_flashattention_fwd_gb300 import cache as fc
import test_cache_cpu as abi
from test_cache_cpu import FakeCuda, lib, make_cache, on  # noqa: F401


@pytest.fixture
def host(monkeypatch):
    """The binding with the launch left out and its allocations on the host."""
    calls = []
    monkeypatch.setattr(fc, "_launch", lambda fn, index, current, args: calls.append(args))
    monkeypatch.setattr(fc, "_current", lambda index: 5)
    monkeypatch.setattr(fc, "_capturing", lambda: False)
    monkeypatch.setattr(fc, "_workspace", lambda *a: (None, 0, 0))
    monkeypatch.setattr(fc.KVCache, "device", property(lambda self: torch.device("cpu")))
    return calls


def evict(cache):
    return fc.cache_evict(cache, on((2, 2, 48), torch.float32), on((2, 2, 48), torch.int32), 20)


def test_new_lengths_are_ordinary_tensors(host, lib):  # noqa: F811
    """The lengths that an eviction returns have nothing in common with those of other calls: not the mode that
    another call ran under, not a version counter, not storage."""
    cache = make_cache()
    with torch.inference_mode():
        inner = evict(cache)
    assert inner.is_inference()
    a, b = evict(cache), evict(cache)
    assert not a.is_inference() and not b.is_inference()
    a.fill_(1).add_(1)                                           # an inference tensor cannot be changed here
    x = torch.ones(4, requires_grad=True)
    y = (x[b.fill_(0).long()] * 2).sum() + x.index_select(0, b).sum()
    a.add_(1)                                                    # b is saved as an index: its counter must not move
    y.backward()
    assert torch.equal(x.grad, torch.tensor([6.0, 0, 0, 0]))
    f = io.BytesIO()
    torch.save(b, f)
    alone = io.BytesIO()
    torch.save(b.clone(), alone)
    assert len(f.getvalue()) == len(alone.getvalue()) and b.untyped_storage().nbytes() == 8


@pytest.mark.parametrize("name", ["k", "v", "seq_len", "table"])
def test_a_cache_keeps_its_tensors(name):
    """A tensor assigned in the place of one that the cache was made with would be passed over in silence: refused.
    What is changed in place is what the calls see, whichever way it is written."""
    cache = make_cache()
    before = getattr(cache, name)
    with pytest.raises(AttributeError, match=name):
        setattr(cache, name, before.clone())
    assert getattr(cache, name) is before
    cache.seq_len += 3
    assert cache.seq_len.tolist() == [3, 3] and fc._PACK(cache.k.data_ptr(), cache.v.data_ptr(), cache.table.data_ptr(),
                                                         cache.seq_len.data_ptr(), 2, 2, 64, 16, 3, 6, 0) == cache._c


@pytest.mark.parametrize("name", ["cache_device.cuh", "cache_schedule.h", "cache_sm103.cu", "tree_sm103.cu", "weigh_sm103.cu"])
def test_overlapped_kernels_load_coherently(name):
    """The cache kernels run while the kernel before them ends.  A non-coherent load asks for data that nobody writes
    while the kernel that reads it runs, which what that kernel leaves behind is not."""
    with open(os.path.join(fa_build.CSRC, name)) as f:
        code = re.sub(r"//.*", "", f.read())
    assert not re.search(r"__ldg|\.nc\b|__restrict__", code)


@pytest.mark.parametrize("call", ["tree", "append", "weights", "evict"])
def test_capacities_that_loops_cannot_step_over_are_refused(lib, call):  # noqa: F811
    """A loop over the slots goes past a sequence's end by up to its step before it stops: the sum has to fit 32 bits."""
    assert getattr(abi, call)(lib, page=64, max_pages=0x7fffff00 // 64) == 2      # 255 below 2^31
    assert getattr(abi, call)(lib, page=64, max_pages=(0x7fffffff - 1024) // 64 + 1) == 2


def test_a_cache_kernel_is_nothing_to_the_others():
    """A change to the cache's kernels leaves the sources of the other kernels alone, and so what was measured of them:
    their status words meet in the host API only."""
    for name in ("fa_fwd_sm103.cu", "fa_fwd1_sm103.cu", "gemm_sm103.cu", "softmax_sm103.cu", "fa_internal.h", "ptx.cuh", "watchdog.cuh"):
        with open(os.path.join(fa_build.CSRC, name)) as f:
            assert not re.search("cache_internal|cache_status|tree_status|weigh_status", f.read()), name


@pytest.mark.parametrize("call,over,words", [
    ("tree", dict(bytes=1000), ["workspace"]), ("tree", dict(scale=-1.0), ["positive"]), ("tree", dict(page=24), ["page", "16"]),
    ("append", dict(weight=abi.ADDR["pos"]), ["written", "overlaps"]), ("evict", dict(first=50, last=51), ["first", "last", "keep"]),
    ("weights", dict(T=0), ["T == 0"]), ("weights", dict(lse=abi.ADDR["lse"] + 2), ["4-byte"])])
def test_messages_name_what_is_wrong(lib, call, over, words):  # noqa: F811
    """The message of a refused call is about that call, not about the forward's arguments alone."""
    message = lib.fa_strerror(getattr(abi, call)(lib, **over)).decode()
    assert all(w in message for w in words), message


@pytest.mark.parametrize("name", ["cache_schedule.h", "cache_sm103.cu", "tree_sm103.cu", "weigh_sm103.cu"])
def test_the_number_of_sms_is_the_device_s(name):
    """Launch shapes follow the device that the call runs on, not the 152 SMs of the one that they were measured on."""
    with open(os.path.join(fa_build.CSRC, name)) as f:
        assert not re.search(r"\b(152|304)\b", re.sub(r"//.*", "", f.read()))


def test_a_copied_cache_is_one_of_its_tensors(monkeypatch):
    """A copy's calls work on the copy's own tensors: the same ones for a shallow copy, others for a deep one."""
    monkeypatch.setattr(FakeCuda, "__deepcopy__", lambda self, memo: memo.setdefault(id(self), on(self.shape, self.dtype)))
    cache = make_cache()
    assert copy.copy(cache)._c == cache._c and copy.copy(cache).seq_len is cache.seq_len
    other = copy.deepcopy({"layers": [cache, make_cache(seq_len=cache.seq_len)]})["layers"]
    for c in other:
        assert c._c == fc._PACK(c.k.data_ptr(), c.v.data_ptr(), c.table.data_ptr(), c.seq_len.data_ptr(), 2, 2, 64, 16, 3, 6, 0)
        assert c.k.data_ptr() != cache.k.data_ptr() and c.seq_len is other[0].seq_len
