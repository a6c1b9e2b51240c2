"""Calls of the cache operators as a user's program makes them: the README's loop over layers, calls that follow one
another with nothing between, calls in forked captures."""
import os
import re

import numpy as np
import pytest
import torch

from test_cache_gpu import fa, ints, normal, pytestmark  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def layer(g, B, Hq, Hkv, D, T, pages, page, cap):
    """One layer's pools, new tokens, weights and positions."""
    pos = torch.arange(cap, dtype=torch.int32).expand(B, Hkv, cap).contiguous()
    return dict(k=normal(g, (pages, Hkv, page, D), "bf16").cuda(), v=normal(g, (pages, Hkv, page, D), "bf16").cuda(),
                q=normal(g, (B, Hq, T, D), "bf16").cuda(), kn=normal(g, (B, Hkv, T, D), "bf16").cuda(),
                vn=normal(g, (B, Hkv, T, D), "bf16").cuda(), weight=torch.rand(B, Hkv, cap, generator=g).cuda(), pos=pos.cuda())


def test_the_readme_s_loop(fa):  # noqa: F811
    """The README's decoding step as it stands there, over three layers: each layer's cache ends as it does when the
    layer is alone (its own lengths, waits between the calls), and every layer evicts."""
    with open(os.path.join(ROOT, "README.md")) as f:
        block, = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "cache_evict" in b]
    g = torch.Generator().manual_seed(110)
    B, Hq, Hkv, D, T, page, n = 2, 4, 2, 64, 5, 64, [4300, 4095]
    per = -(-(n[0] + T) // page)
    table = torch.randperm(B * per + 1, generator=g)[:B * per].reshape(B, per)
    parent, path, count = [[-1, 0, 1, 1, 0]] * B, [[0, 1, 3, -1, -1], [0, 4, -1, -1, -1]], [3, 2]
    layers = [layer(g, B, Hq, Hkv, D, T, B * per + 1, page, per * page) for _ in range(3)]
    alone = [{x: t.clone() for x, t in a.items()} for a in layers]
    L = {x: [a[x] for a in layers] for x in layers[0]}
    env = dict(pools=list(zip(L["k"], L["v"])), seq_len=ints(n), table=ints(table), q=L["q"], k_new=L["kn"], v_new=L["vn"], o=[None] * 3,
               lse=[None] * 3, parent=ints(parent), path=ints(path), count=ints(count), weight=L["weight"], pos=L["pos"], next_pos=ints(n))
    exec(compile(block, "README.md", "exec"), env)
    assert env["seq_len"].tolist() == [4096, 4096] and env["next_pos"].tolist() == [4303, 4097]
    for a, b in zip(layers, alone):
        cache = fa.KVCache(b["k"], b["v"], ints(n), ints(table))
        torch.cuda.synchronize()
        _, lse = fa.tree_attention(b["q"], b["kn"], b["vn"], cache, parent=ints(parent))
        torch.cuda.synchronize()
        fa.cache_append(cache, b["kn"], b["vn"], path=ints(path), count=ints(count), weight=b["weight"], pos=b["pos"], start=ints(n))
        cache.seq_len.add_(ints(count))
        torch.cuda.synchronize()
        fa.cache_weights(cache, b["q"], lse, b["weight"], path=ints(path), count=ints(count))
        torch.cuda.synchronize()
        moved = b["pos"].clone()
        fa.cache_evict(cache, b["weight"], b["pos"], keep=4096, first=4, last=512, next_pos=ints(np.add(n, count)))
        torch.cuda.synchronize()
        assert all((moved[x] != b["pos"][x]).any() for x in range(B))
        for x in ("k", "v", "weight", "pos"):
            assert torch.equal(a[x], b[x]), x
