"""Calls of the cache operators as a user's program makes them: the README's loop over layers, calls that follow one
another with nothing between, calls in forked captures."""
import os
import re

import numpy as np
import pytest
import torch

from test_cache_gpu import debug_call, fa, ints, normal, pytestmark  # noqa: F401

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


def test_calls_with_nothing_between(fa):  # noqa: F811
    """Attention, its weights (causal=False: before the append) and an eviction by them, one behind the other, so that each
    starts while the one before ends and reads what that one writes: lse, weights, rows.  New queries every time, in the
    same buffers, against the same calls with a wait behind each."""
    g = torch.Generator().manual_seed(120)
    B, Hq, Hkv, D, T, page, n, keep = 8, 8, 2, 128, 6, 64, 700, 650
    per = -(-(n + T) // page)
    table = ints(torch.randperm(B * per, generator=g).reshape(B, per))
    a = layer(g, B, Hq, Hkv, D, T, B * per, page, per * page)
    b = {x: t.clone() for x, t in a.items()}
    path, count = ints([[0, 2, 3, -1, -1, -1]] * B), ints([3] * B)

    def step(c, wait):
        cache = c["cache"]
        fa.tree_attention(c["q"], c["kn"], c["vn"], cache, o=c["o"], lse=c["lse"])
        wait()
        fa.cache_weights(cache, c["q"], c["lse"], c["weight"], path=path, count=count, causal=False)
        wait()
        fa.cache_evict(cache, c["weight"], c["pos"], keep, first=2, last=20, next_pos=c["next"], new_len=c["seq"])
        wait()
        fa.tree_attention(c["q"], c["kn"], c["vn"], cache, o=c["o2"], lse=c["lse2"])
        wait()
        fa.cache_append(cache, c["kn"], c["vn"], path=path, count=count, weight=c["weight"], pos=c["pos"], start=c["next"])
        wait()
        return [c[x] for x in ("o", "lse", "weight", "pos", "k", "v", "o2", "lse2", "seq")]

    for c in (a, b):
        c.update(seq=ints([n] * B), next=ints([n] * B), o=torch.zeros_like(c["q"]), lse=torch.zeros(B, Hq, T, device="cuda"))
        c.update(o2=torch.zeros_like(c["q"]), lse2=torch.zeros_like(c["lse"]), len=ints([n] * B))
        c["cache"] = fa.KVCache(c["k"], c["v"], c["len"], table)
    for _ in range(12):
        q = normal(g, tuple(a["q"].shape), "bf16").cuda()
        for c in (a, b):
            c["q"].copy_(q)
            c["len"].fill_(n)
        torch.cuda.synchronize()
        got = step(a, lambda: None)
        want = step(b, torch.cuda.synchronize)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), i
        assert a["seq"].tolist() == [keep] * B


def test_a_forked_capture(fa):  # noqa: F811
    """Two layers' attention on two streams of one capture, joined before what reads both; replayed with new queries."""
    g = torch.Generator().manual_seed(130)
    B, Hq, Hkv, D, T, page, n = 2, 8, 2, 64, 4, 32, 500
    per = -(-n // page)
    table = ints(torch.randperm(B * per, generator=g).reshape(B, per))
    layers = [layer(g, B, Hq, Hkv, D, T, B * per, page, per * page) for _ in range(2)]
    seq = ints([n, n - 37])
    caches = [fa.KVCache(c["k"], c["v"], seq, table) for c in layers]

    def calls(fork):
        main, other, out = torch.cuda.current_stream(), torch.cuda.Stream() if fork else torch.cuda.current_stream(), []
        if fork:
            other.wait_stream(main)
        for s, c, cache in zip((main, other), layers, caches):
            with torch.cuda.stream(s):
                out += fa.tree_attention(c["q"], c["kn"], c["vn"], cache)
        if fork:
            main.wait_stream(other)
        for i, (c, cache) in enumerate(zip(layers, caches)):
            out.append(fa.cache_weights(cache, c["q"], out[2 * i + 1], c["weight"], causal=False, out=torch.zeros_like(c["weight"])))
        return out

    calls(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(True)
    for _ in range(4):
        for c in layers:
            c["q"].copy_(normal(g, tuple(c["q"].shape), "bf16"))
        seq.copy_(ints([n - 10, n]))
        want = calls(False)
        torch.cuda.synchronize()
        for x in got:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for c, i in zip(layers, (4, 5)):
            got[i].masked_fill_(got[i] == 7, 0)        # slots that are not in use are left as they were
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 4), (128, 80), (256, 4)])
def test_ctas_without_room(fa, D, Hq):  # noqa: F811
    """CTAs that act as if their shared memory were too small: the call ends, the status says so, every row is NaN, those of
    units that are joined from parts too (the workspace holds nothing that the joining kernel may go by), rows
    behind draft_len are as they were, and the next call is right.  (Hq = 80: two row tiles side by side.)"""
    g = torch.Generator().manual_seed(140)
    B, Hkv, T, page, n = 12, 2, 5, 64, 1500
    per = -(-n // page)
    c = layer(g, B, Hq, Hkv, D, T, B * per, page, per * page)
    cache = fa.KVCache(c["k"], c["v"], ints([n] * B), ints(torch.arange(B * per).reshape(B, per)))
    drafts = ints([5, 4, 0] * 4)
    want = fa.tree_attention(c["q"], c["kn"], c["vn"], cache, draft_len=drafts, o=torch.full_like(c["q"], 7), lse=torch.full((B, Hq, T), 9.0).cuda())
    o, lse = torch.full_like(c["q"], 7), torch.full((B, Hq, T), 9.0, device="cuda")
    size = fa.tree_workspace_bytes(Hq, Hkv, T, D)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    debug_call(fa, "fa_tree_debug", cache, (c["q"], c["kn"], c["vn"], None, drafts, o, lse),
               (Hq, T, D ** -0.5, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream, 0, 4))
    st, word = fa.fa_device_status()
    assert st == 12 and word & 0xff01 == 0x901
    live = torch.arange(T, device="cuda") < drafts[:, None, None]
    live = live.expand(B, Hq, T)
    assert torch.isnan(o[live]).all() and torch.isnan(lse[live]).all() and (o[~live] == 7).all() and (lse[~live] == 9).all()
    again = fa.tree_attention(c["q"], c["kn"], c["vn"], cache, draft_len=drafts, o=o, lse=lse)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1]) and fa.fa_device_status() == (0, 0)


def test_one_call_reads_the_words_of_all_kernels(fa):  # noqa: F811
    """Attention and weights that both gave up before anyone asked: reported once, both words cleared."""
    g = torch.Generator().manual_seed(150)
    B, Hq, Hkv, D, T, page, n = 2, 4, 2, 64, 3, 16, 300
    per = -(-n // page)
    c = layer(g, B, Hq, Hkv, D, T, B * per, page, per * page)
    cache = fa.KVCache(c["k"], c["v"], ints([n] * B), ints(torch.arange(B * per).reshape(B, per)))
    o, lse, out = torch.zeros_like(c["q"]), torch.zeros(B, Hq, T, device="cuda"), torch.zeros_like(c["weight"])
    ws = torch.zeros(max(fa.tree_workspace_bytes(Hq, Hkv, T, D), fa.weights_workspace_bytes()), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    debug_call(fa, "fa_tree_debug", cache, (c["q"], c["kn"], c["vn"], None, None, o, lse),
               (Hq, T, D ** -0.5, ws.data_ptr(), ws.nbytes, stream, 3_000_000, 1))
    debug_call(fa, "fa_weights_debug", cache, (c["q"], lse, None, None, None, out),
               (Hq, T, 1, D ** -0.5, ws.data_ptr(), ws.nbytes, stream, 3_000_000, 1))
    st, word = fa.fa_device_status()
    assert st == 12 and word & 1 and torch.isnan(lse).all() and torch.isnan(out[..., :n]).all()
    assert fa.fa_device_status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 4), (64, 96), (128, 96), (256, 4)])
def test_a_non_finite_value_in_use_is_not_lost(fa, dtype, D, Hq):  # noqa: F811
    """An infinity in a cached value that every row sees, with a weight of e^-240 (0 in 32 bits): the result is not finite
    there, wherever the keys are cut (many equal sequences: in every place), and right everywhere else."""
    g = torch.Generator().manual_seed(160)
    B, Hkv, T, page, n, per = 40, 2, 3, 64, 200, 4
    c = layer(g, B, Hq, Hkv, D, T, B * per, page, per * page)
    k, v, q, kn, vn = (c[x].to(torch.bfloat16 if dtype == "bf16" else torch.float16) for x in ("k", "v", "q", "kn", "vn"))
    q[..., 0], kn[..., 0] = D ** 0.5, 0
    k[..., 0] = 0
    k[2::per, ..., 0], k[3::per, ..., 0] = 240, 240              # slots from 128 on: a later key step
    cache = fa.KVCache(k, v, ints([n] * B), ints(torch.arange(B * per).reshape(B, per)))
    want, want_lse = fa.tree_attention(q, kn, vn, cache)
    v[0::per, :, 7, 5] = float("inf")                            # slot 7
    o, lse = fa.tree_attention(q, kn, vn, cache)
    assert torch.isfinite(want).all() and not torch.isfinite(o[..., 5]).any()
    rest = [d for d in range(D) if d != 5]
    assert torch.equal(o[..., rest], want[..., rest]) and torch.equal(lse, want_lse)


def test_calls_with_nothing_to_do(fa):  # noqa: F811
    """No drafted, counted or cached token in any sequence: nothing is written but the lengths."""
    g = torch.Generator().manual_seed(170)
    B, Hq, Hkv, D, T, page = 3, 4, 2, 128, 5, 16
    c = layer(g, B, Hq, Hkv, D, T, B * 4, page, 4 * page)
    seq, none = ints([0, 20, 33]), ints([0, 0, -2])
    cache = fa.KVCache(c["k"], c["v"], seq, ints(torch.arange(B * 4).reshape(B, 4)))
    before = {x: t.clone() for x, t in c.items()}
    o, lse = fa.tree_attention(c["q"], c["kn"], c["vn"], cache, draft_len=none, o=torch.full_like(c["q"], 7), lse=torch.full((B, Hq, T), 9.0).cuda())
    assert (o == 7).all() and (lse == 9).all()
    fa.cache_append(cache, c["kn"], c["vn"], count=none, weight=c["weight"], pos=c["pos"], start=seq)
    for T2 in (5, 200):                                          # packed rows, and the tiles of a prompt
        q, l = torch.full((B, Hq, T2, D), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((B, Hq, T2), float("nan"), device="cuda")
        fa.cache_weights(cache, q, l, c["weight"], count=none)
    fa.cache_weights(cache, q, l, c["weight"], path=ints(torch.zeros(B, 200)), count=none)
    seq.zero_()
    fa.cache_weights(cache, q, l, c["weight"])
    assert fa.cache_evict(cache, c["weight"], c["pos"], 4).tolist() == [0, 0, 0]
    for x in before:
        assert torch.equal(c[x], before[x]), x
    assert fa.fa_device_status() == (0, 0)


@pytest.mark.parametrize("which", ["weight_out", "pos_out"])
def test_evict_with_one_of_its_results_elsewhere(fa, which):  # noqa: F811
    g = torch.Generator().manual_seed(180)
    B, Hkv, D, page, n, keep = 2, 2, 64, 16, 500, 333
    per = -(-n // page)
    c = layer(g, B, 4, Hkv, D, 1, B * per, page, per * page)
    outs, kept = [], []
    for other in (False, True):
        k, v, w, p = (c[x].clone() for x in ("k", "v", "weight", "pos"))
        cache = fa.KVCache(k, v, ints([n, n - 3]), ints(torch.arange(B * per).reshape(B, per)))
        given = {which: torch.zeros_like(w if which == "weight_out" else p)} if other else {}
        fa.cache_evict(cache, w, p, keep, first=2, last=9, next_pos=ints([n, n - 3]), **given)
        outs.append([x[..., :keep] for x in (given.get("weight_out", w), given.get("pos_out", p))] + [k, v])
        kept.append((w, p))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    same = 0 if which == "weight_out" else 1                     # the one whose result went elsewhere is as it was
    assert torch.equal(kept[1][same], c["weight" if same == 0 else "pos"])


def test_evict_with_more_protected_slots_than_it_keeps(fa):  # noqa: F811
    """Positions at or above next_pos, or the same one again and again: the lowest protected slots stay, in order."""
    g = torch.Generator().manual_seed(190)
    B, Hkv, D, page, n, keep = 2, 2, 64, 16, 3000, 700
    per = -(-n // page)
    c = layer(g, B, 4, Hkv, D, 1, B * per, page, per * page)
    safe = torch.rand(B, Hkv, per * page, generator=g) < 0.5
    pos = torch.where(safe, torch.where(torch.rand(safe.shape, generator=g) < 0.3, 1, n + 5), n - 200).to(torch.int32)
    k, v, w, p = c["k"].clone(), c["v"].clone(), c["weight"].clone(), pos.cuda()
    fa.cache_evict(fa.KVCache(k, v, ints([n] * B), ints(torch.arange(B * per).reshape(B, per))), w, p, keep, first=2, last=9, next_pos=ints([n] * B))
    K, V = (x.reshape(B, per, Hkv, page, D).transpose(1, 2).reshape(B, Hkv, -1, D) for x in (c["k"], c["v"]))
    K2, V2 = (x.reshape(B, per, Hkv, page, D).transpose(1, 2).reshape(B, Hkv, -1, D) for x in (k, v))
    for b in range(B):
        for h in range(Hkv):
            kept = torch.nonzero(safe[b, h, :n])[:keep, 0]
            slots = torch.arange(keep)
            slots[~safe[b, h, :keep]] = kept[kept >= keep]
            slots = slots.cuda()
            assert torch.equal(w[b, h, :keep], c["weight"][b, h, slots]) and torch.equal(p[b, h, :keep].cpu(), pos[b, h, slots.cpu()])
            assert torch.equal(K2[b, h, :keep], K[b, h, slots]) and torch.equal(V2[b, h, :keep], V[b, h, slots])


@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (256, 32)])
def test_what_the_lengths_do_not_cover_is_not_used(fa, D, page):  # noqa: F811
    """Table entries behind a sequence's pages, drafted rows behind draft_len and their parents, path entries behind count,
    weights and positions behind seq_len hold anything: the results are those with clean ones."""
    g = torch.Generator().manual_seed(200 + D)
    B, Hq, Hkv, T, per, n, drafts, counts = 4, 8, 2, 9, 40, [0, 1, 500, 37], [9, 0, 4, 7], [2, 0, 3, 7]
    c = layer(g, B, Hq, Hkv, D, T, B * per, page, per * page)
    parent, path = torch.tensor([[-1, 0, 1, 1, 0, 4, 2, 6, 7]] * B), torch.arange(T).repeat(B, 1)
    clean = torch.arange(B * per).reshape(B, per)
    results = []
    for dirty in (False, True):
        x = {k: t.clone() for k, t in c.items()}
        table, par, way, seq = clean.clone(), parent.clone(), path.clone(), ints(n)
        if dirty:
            for b in range(B):
                table[b, -(-(n[b] + counts[b]) // page):] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31, 7])[torch.randint(0, 4, (1,), generator=g)]
                par[b, drafts[b]:], way[b, counts[b]:] = 2 ** 31 - 1, -2 ** 31
                x["q"][b, :, drafts[b]:], x["kn"][b, :, drafts[b]:], x["vn"][b, :, drafts[b]:] = float("nan"), float("inf"), float("nan")
                x["weight"][b, :, n[b] + counts[b]:], x["pos"][b, :, n[b] + counts[b]:] = float("nan"), -2 ** 31
        cache = fa.KVCache(x["k"], x["v"], seq, ints(table))
        o, lse = fa.tree_attention(x["q"], x["kn"], x["vn"], cache, parent=ints(par), draft_len=ints(drafts), o=torch.full_like(x["q"], 7),
                                   lse=torch.full((B, Hq, T), 9.0, device="cuda"))
        kept = lse.clone()
        if dirty:
            for b in range(B):
                kept[b, :, drafts[b]:] = float("nan")
        fa.cache_append(cache, x["kn"], x["vn"], path=ints(way), count=ints(counts), weight=x["weight"], pos=x["pos"], start=seq.clone())
        seq += ints(counts)
        fa.cache_weights(cache, x["q"], kept, x["weight"], path=ints(way), count=ints(counts))
        left = fa.cache_evict(cache, x["weight"], x["pos"], 30, first=2, last=5, next_pos=seq)
        live = [(x["weight"][b, :, :m], x["pos"][b, :, :m]) for b, m in enumerate(left.tolist())]
        results.append([o, lse, x["k"], x["v"], left] + [t for pair in live for t in pair])
    assert fa.fa_device_status() == (0, 0)
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b), i
