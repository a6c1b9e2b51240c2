"""GPU tests of the rotary operators against their definition in float64.

Tolerances, from the arithmetic.  u = eps / 2 is the type's rounding (2^-8 bf16, 2^-11 fp16).  The fraction of a turn is exact to 2^-32
and rounded to 24 bits as an fp32 argument of sincospif (an angle off by at most pi 2^-25 < 2^-23), which is within 2 units
of the last place (2^-23); the amplitude and the two products add 2^-24 each:
    |y - ref| <= 2^-20 amplitude (|a| + |b|) + u |ref|,   in fp16 half a step of 2^-25 below the normal range.
What is not rotated is copied: equal.
"""
import copy
import os
import re

import numpy as np
import pytest
import torch

from test_cache_gpu import DT, U, fa, ints, pytestmark  # noqa: F401


def turned(x, table, position, inverse=False):
    """(y, tolerance) in float64; x [B, H, T, D], position [B, T]."""
    x = x.detach().double().cpu().numpy()
    rot, f = table.rot, np.array(table.frequencies)
    t = np.asarray(position, np.float64)[:, None, :, None] * f
    c, s = np.cos(t) * table.amplitude, np.sin(t) * table.amplitude * (-1 if inverse else 1)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if table.interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, tol = x.copy(), np.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    size = abs(table.amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol[..., a] = tol[..., b] = 2.0 ** -20 * size
    return y, tol


def near(got, ref, dtype, rot):
    y, tol = ref
    d = np.abs(got.detach().double().cpu().numpy() - y)
    tol = tol + U[dtype] * np.abs(y) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert (d <= tol).all(), (np.argwhere(d > tol)[0], d.max())
    assert (d[..., rot:] == 0).all()


def data(seed, dtype, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


TURNS = [(64, 64, False), (64, 32, True), (128, 128, True), (128, 96, False), (128, 50, False), (128, 50, True), (256, 256, False), (256, 64, True),
         (64, 0, False), (64, 2, True), (64, 18, False)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("turn", TURNS, ids=str)
def test_rotary(fa, turn, dtype):  # noqa: F811
    """Dense tensors and the rows of one projection, positions by t, by start and by a table of far and negative ones."""
    D, rot, inter = turn
    table = fa.RotaryTable(D, rot=rot, interleaved=inter, amplitude=1.25)
    for B, Hq, Hk, T in ((1, 1, 1, 1), (3, 5, 2, 37), (2, 8, 8, 130)):
        q, k = data(1, dtype, B, Hq, T, D), data(2, dtype, B, Hk, T, D)
        at = np.arange(T)[None].repeat(B, 0)
        yq, yk = fa.rotary(table, q, k)
        near(yq, turned(q, table, at), dtype, rot)
        near(yk, turned(k, table, at), dtype, rot)
        r = np.random.default_rng(3)
        start = r.integers(-1000, 2 ** 20, B)
        assert torch.equal(fa.rotary(table, q, start=ints(start)), fa.rotary(table, q, position=ints(start[:, None] + at)))
        far = r.integers(-2 ** 31, 2 ** 31, (B, T))
        near(fa.rotary(table, q, position=ints(far), inverse=True), turned(q, table, far, True), dtype, rot)
        fused = data(4, dtype, B, T, (Hq + 2 * Hk) * D)
        heads = fused.view(B, T, Hq + 2 * Hk, D).transpose(1, 2)
        before = fused.clone()
        yq, yk = fa.rotary(table, heads[:, :Hq], heads[:, Hq:Hq + Hk], start=ints(start))
        assert torch.equal(fused, before)
        near(yq, turned(heads[:, :Hq], table, start[:, None] + at), dtype, rot)
        near(yk, turned(heads[:, Hq:Hq + Hk], table, start[:, None] + at), dtype, rot)
        # in place, in the projection's rows; what is neither query nor key stays
        a, b = heads[:, :Hq], heads[:, Hq:Hq + Hk]
        got = fa.rotary(table, a, b, start=ints(start), q_out=a, k_out=b)
        assert got[0] is a and got[1] is b and torch.equal(a, yq) and torch.equal(b, yk)
        assert torch.equal(heads[:, Hq + Hk:], before.view(B, T, Hq + 2 * Hk, D).transpose(1, 2)[:, Hq + Hk:])


def test_exact_angles_far_away(fa):  # noqa: F811
    """The fastest pair at positions up to 2^31 - 1: an fp32 angle would be off by up to 64 radians there."""
    table = fa.RotaryTable(64)
    far = np.array([[0, 1, 65535, 65536, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31]])
    x = torch.zeros(1, 1, 8, 64, device="cuda", dtype=torch.float16)
    x[..., 0] = 1
    y = fa.rotary(table, x, position=ints(far)).double().cpu().numpy()[0, 0]
    assert np.abs(y[:, 0] - np.cos(far[0].astype(np.float64))).max() <= 2.0 ** -11 and np.abs(y[:, 32] - np.sin(far[0].astype(np.float64))).max() <= 2.0 ** -11


def test_many_heads_and_tokens(fa):  # noqa: F811
    """Threads that go through several heads, in uneven runs, across the border of queries and keys."""
    table = fa.RotaryTable(128, scaling="ramp", factor=8.0, original=4096)
    q, k = data(5, "bf16", 2, 33, 6001, 128), data(6, "bf16", 2, 11, 6001, 128)
    yq, yk = fa.rotary(table, q, k)
    at = np.arange(6001)[None].repeat(2, 0)
    for h in (0, 15, 31, 32):
        near(yq[:, h:h + 1], turned(q[:, h:h + 1], table, at), "bf16", 128)
    for h in (0, 5, 10):
        near(yk[:, h:h + 1], turned(k[:, h:h + 1], table, at), "bf16", 128)


def test_values_that_are_not_rotated(fa):  # noqa: F811
    """NaN and infinities behind rot are copied bit by bit, and touch nothing else; position 0 copies everything."""
    table = fa.RotaryTable(64, rot=32)
    x = data(7, "bf16", 1, 2, 9, 64)
    clean = fa.rotary(table, x, start=ints([5]))
    x[..., 32:] = float("nan")
    x[..., 40] = -float("inf")
    y = fa.rotary(table, x, start=ints([5]))
    assert torch.equal(y[..., :32], clean[..., :32]) and torch.equal(y[..., 32:].view(torch.int16), x[..., 32:].view(torch.int16))
    x = data(8, "fp16", 1, 2, 1, 64)
    assert torch.equal(fa.rotary(table, x), x)


def test_inverse_is_the_gradient(fa):  # noqa: F811
    """<R x, g> = <x, R^T g>, and the inverse of the rotation undoes it up to the amplitude's square."""
    table = fa.RotaryTable(128, rot=64, interleaved=True, amplitude=1.25)
    x, g = data(9, "fp16", 2, 3, 50, 128), data(10, "fp16", 2, 3, 50, 128)
    y, back = fa.rotary(table, x, start=ints([3, 70000])), fa.rotary(table, g, start=ints([3, 70000]), inverse=True)
    left, right = (y.double() * g.double()).sum(), (x.double() * back.double()).sum()
    # each product is off by a rounding of its factor: 2 u sum |y||g| in all, both sides
    assert (left - right).abs() <= 4 * U["fp16"] * (y.double().abs() * g.double().abs()).sum()
    again = fa.rotary(table, y, start=ints([3, 70000]), inverse=True).double()
    want = x.double().clone()
    want[..., :64] *= 1.25 ** 2
    assert ((again - want).abs() <= 2.0 ** -8 * (1 + want.abs())).all()   # 1.25 (|da| + |db|) + u |y|, each da <= u 1.25 (|a| + |b|), |a|, |b| <= 5


def test_autograd(fa):  # noqa: F811
    table = fa.RotaryTable(64, rot=32)
    fused = data(11, "bf16", 2, 20, 6 * 64).requires_grad_()
    heads = fused.view(2, 20, 6, 64).transpose(1, 2)
    q, k = fa.rotary_ad(table, heads[:, :4], heads[:, 4:], start=ints([0, 9]))
    gq, gk = data(12, "bf16", 2, 4, 20, 64), data(13, "bf16", 2, 2, 20, 64)
    torch.autograd.backward((q, k), (gq, gk))
    want = torch.cat(fa.rotary(table, gq, gk, start=ints([0, 9]), inverse=True), 1)
    assert torch.equal(fused.grad.view(2, 20, 6, 64).transpose(1, 2), want)
    x = data(14, "bf16", 1, 2, 3, 64).requires_grad_()
    fa.rotary_ad(table, x).sum().backward()     # an expanded gradient
    assert torch.equal(x.grad, fa.rotary(table, torch.ones_like(x), inverse=True))


def test_copies_of_a_table(fa):  # noqa: F811
    table = fa.RotaryTable(64, rot=32, scaling="linear", factor=3.0, amplitude=0.5)
    twin = copy.deepcopy(table)
    x = data(15, "bf16", 1, 2, 30, 64)
    assert twin.freq.data_ptr() != table.freq.data_ptr() and torch.equal(twin.freq, table.freq) and torch.equal(fa.rotary(twin, x), fa.rotary(table, x))


# ---------------------------------------------------------------- with the cache's writes

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,Hq,Hkv,D,T,page,turn", [(1, 4, 2, 128, 1, 64, (128, False)), (3, 6, 3, 64, 21, 16, (32, True)), (2, 2, 2, 256, 100, 48, (250, False)),
                                                    (4, 0, 2, 64, 9, 32, (64, True))], ids=str)
def test_append(fa, B, Hq, Hkv, D, T, page, turn, dtype):  # noqa: F811
    """Ragged counts (none, all, more than all), lengths that end inside a page, a page that does not exist, a sequence at its
    capacity: results, slots, weights and positions as defined, everything else as it was."""
    table = fa.RotaryTable(D, rot=turn[0], interleaved=turn[1])
    g = torch.Generator().manual_seed(1)
    per = -(-(40 + T) // page) + 1
    pages = torch.randperm(B * per + 2, generator=g)[:B * per].reshape(B, per)
    k_pool, v_pool = data(1, dtype, B * per + 2, Hkv, page, D), data(2, dtype, B * per + 2, Hkv, page, D)
    cap = per * page
    lens = [40, cap - 5, 0, 17][:B]
    count = [T, T, 0, T + 3][:B] if B > 1 else [T]
    if B > 2:
        pages[2, 0] = -1
    if B > 3:
        pages[3, 17 // page] = 10 ** 6
    fused = data(3, dtype, B, T, (Hq + 2 * Hkv) * D)
    heads = fused.view(B, T, Hq + 2 * Hkv, D).transpose(1, 2)
    q, k, v = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
    start = np.array([7, 100000, 5, 0][:B])
    weight, pos = torch.rand(B, Hkv, cap, device="cuda"), torch.full((B, Hkv, cap), -7, dtype=torch.int32, device="cuda")
    for how in (dict(start=ints(start)), dict(position=ints(start[:, None] + np.arange(T))), dict()):
        base = np.array(lens) if not how else start
        kp, vp, w, ps = k_pool.clone(), v_pool.clone(), weight.clone(), pos.clone()
        out = [torch.full((B, h, T, D), 3.0, dtype=DT[dtype], device="cuda") for h in (Hq, Hkv, Hkv)]
        cache = fa.KVCache(kp, vp, ints(lens), ints(pages))
        got = fa.rotary_append(cache, table, q, k, v, count=ints(count), weight=w, pos=ps, q_out=out[0], k_out=out[1], v_out=out[2], **how)
        assert all(x is y for x, y in zip(got, out))
        at = base[:, None] + np.arange(T)
        yq, yk = fa.rotary(table, q, k, position=ints(at))   # tested above
        wk, wv, ww, wp = k_pool.clone(), v_pool.clone(), weight.clone(), pos.clone()
        want = [torch.full_like(x, 3.0) for x in out]
        for b in range(B):
            n = min(count[b], T)
            for x, y in zip(want, (yq, yk, v)):
                x[b, :, :n] = y[b, :, :n]
            for i in range(n):
                s = lens[b] + i
                if s >= cap:
                    break
                ww[b, :, s], wp[b, :, s] = 0.0, int(at[b, i])
                pid = int(pages[b, s // page])
                if 0 <= pid < len(k_pool):
                    wk[pid, :, s % page], wv[pid, :, s % page] = yk[b, :, i], v[b, :, i]
        for x, y in zip((*out, kp, vp, w, ps), (*want, wk, wv, ww, wp)):
            assert torch.equal(x, y)
        kp.copy_(k_pool), vp.copy_(v_pool)
        none = fa.rotary_append(cache, table, q, k, v, count=ints(count), k_out=False, v_out=False, **how)
        assert none[1] is None and none[2] is None and torch.equal(kp, wk) and torch.equal(vp, wv)


def test_append_then_attention(fa):  # noqa: F811
    """A decoding loop as it is used: a prompt, then one token at a time, against one causal attention over all of them."""
    B, Hq, Hkv, D, n, steps, page = 2, 8, 2, 128, 70, 4, 32
    table = fa.RotaryTable(D, rot=64)
    total = n + steps
    fused = data(20, "bf16", B, total, (Hq + 2 * Hkv) * D)
    heads = fused.view(B, total, Hq + 2 * Hkv, D).transpose(1, 2)
    q, k, v = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
    yq, yk = fa.rotary(table, q, k)
    ref, ref_lse = fa.attention(yq, yk, v.contiguous(), causal=True)
    per = -(-total // page)
    cache = fa.KVCache(torch.zeros(B * per, Hkv, page, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B * per, Hkv, page, D, dtype=torch.bfloat16, device="cuda"),
                       ints([0] * B), ints(np.random.default_rng(0).permutation(B * per).reshape(B, per)))
    t = slice(0, n)
    a, b, c = fa.rotary_append(cache, table, q[:, :, t], k[:, :, t], v[:, :, t])
    o, lse = fa.attention(a, b, c, causal=True)
    cache.seq_len += n
    assert torch.equal(o, ref[:, :, t])
    for i in range(n, total):
        t = slice(i, i + 1)
        a, b, c = fa.rotary_append(cache, table, q[:, :, t], k[:, :, t], v[:, :, t])
        o, lse = fa.tree_attention(a, b, c, cache)
        cache.seq_len += 1
        # two orders of the same sums: P and o are rounded once in each (u of sum p |v| <= 5, and of o)
        assert (o.double() - ref[:, :, t].double()).abs().max() <= 4 * U["bf16"] * 5 and (lse - ref_lse[:, :, t]).abs().max() <= 2.0 ** -14
    assert torch.equal(cache.k[cache.table.long()].transpose(2, 3).reshape(B, -1, Hkv, D)[:, :total].transpose(1, 2), yk)


def test_streams_and_graphs(fa):  # noqa: F811
    """A call on a stream of its own, and one captured and replayed over other inputs, lengths and positions."""
    table = fa.RotaryTable(64)
    q, k, v = (data(30 + i, "bf16", 2, h, 5, 64) for i, h in enumerate((4, 2, 2)))
    cache = fa.KVCache(torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda"), ints([3, 20]))
    want = fa.rotary(table, q, k, start=ints([3, 20]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.rotary_append(cache, table, q, k, v, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], v)
    graph = torch.cuda.CUDAGraph()
    start = ints([0, 0])
    with torch.cuda.graph(graph):
        y = fa.rotary(table, q, k, start=start)
        z = fa.rotary_append(cache, table, q, k, v, start=start)
    for s in ([5, 9], [1000, 70]):
        q.copy_(data(s[0], "bf16", 2, 4, 5, 64))
        start.copy_(ints(s))
        graph.replay()
        want = fa.rotary(table, q, k, start=ints(s))
        assert all(torch.equal(a, b) for a, b in zip((*y, *z[:2]), want * 2))


def test_binding_refuses(fa):  # noqa: F811
    table = fa.RotaryTable(64)
    x = data(1, "bf16", 1, 2, 4, 64)
    for bad in (lambda: fa.rotary(table, x.float()), lambda: fa.rotary(table, x[..., :32]), lambda: fa.rotary(table, x.cpu()), lambda: fa.rotary(table, x, x.half()),
                lambda: fa.rotary(table, x, start=ints([0]), position=ints([[0] * 4])), lambda: fa.rotary(table, x, start=ints([0, 1])),
                lambda: fa.rotary(table, x, k_out=x), lambda: fa.rotary(table, x.transpose(2, 3).contiguous().transpose(2, 3)),
                lambda: fa.rotary(table, x, q_out=x[:, :1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fa.FaError):   # rows that are not on 16 bytes
        fa.rotary(table, data(1, "bf16", 1, 2, 4, 68)[..., 4:])
    with pytest.raises(TypeError):
        fa.rotary(None, x)


def test_more_than_32_bits_of_elements(fa):  # noqa: F811
    """2.2e9 elements read and written, and a pool of as many: the last heads, tokens and pages are as they are alone."""
    B, H, T, D = 4, 33, 131072, 128
    table = fa.RotaryTable(D)
    x = torch.full((B, T, H, D), 0.5, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    assert x.numel() > 2 ** 31
    tail = data(40, "bf16", 1, 2, 100, D)
    x[-1:, -2:, -100:] = tail
    y = fa.rotary(table, x, start=ints([0, 0, 0, 7]))
    assert torch.equal(y[-1:, -2:, -100:], fa.rotary(table, tail, start=ints([7 + T - 100])))
    del x, y
    Hkv, page = 8, 128
    num = 2 ** 31 // (Hkv * page * D) + 8
    k, v = (torch.zeros(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = fa.KVCache(k, v, ints([3]), ints([[num - 1]]))
    q, kn, vn = (data(41 + i, "bf16", 1, h, 5, D) for i, h in enumerate((8, 8, 8)))
    _, kr, _ = fa.rotary_append(cache, table, q, kn, vn)
    assert torch.equal(k[num - 1, :, 3:8], kr[0]) and torch.equal(v[num - 1, :, 3:8], vn[0])
    assert not k[num - 1, :, 8:].any() and not k[num - 1, :, :3].any() and not k[num - 2].any() and not k[0].any()


def test_calls_with_nothing_between(fa):  # noqa: F811
    """Rotation, append, attention and append again back to back, each reading what the one before writes, over and over in
    the same buffers, against the same calls with a wait behind each."""
    B, Hq, Hkv, D, T, page, n = 4, 8, 2, 64, 3, 16, 60
    table = fa.RotaryTable(D)
    per = -(-(n + 30 * T) // page)

    def make():
        return dict(k=data(50, "bf16", B * per, Hkv, page, D), v=data(51, "bf16", B * per, Hkv, page, D), len=ints([n, 5, 33, 48]),
                    q=torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device="cuda"), kn=torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda"),
                    vn=torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda"), o=torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device="cuda"),
                    rows=torch.zeros(B, T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda"))
    rows = data(52, "bf16", 20, B, T, (Hq + 2 * Hkv) * D)

    def step(c, i, wait):
        cache = fa.KVCache(c["k"], c["v"], c["len"])
        c["rows"].copy_(rows[i])
        h = c["rows"].view(B, T, -1, D).transpose(1, 2)
        fa.rotary_append(cache, table, h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:], q_out=c["q"], k_out=c["kn"], v_out=c["vn"])
        wait()
        fa.tree_attention(c["q"], c["kn"], c["vn"], cache, o=c["o"])
        wait()
        c["len"] += T
        fa.rotary(table, c["o"], start=c["len"], q_out=c["q"])
        wait()
        return c["q"].clone()
    a, b = make(), make()
    got = [step(a, i, lambda: None) for i in range(20)]
    want = [step(b, i, torch.cuda.synchronize) for i in range(20)]
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])


def readme(word):
    """The README's one block of Python that contains `word`."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        block, = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if word in b]
    return compile(block, "README.md", "exec")


def test_the_readme_s_training_step(fa):  # noqa: F811
    """As it stands there, against the same steps one by one; the gradient arrives in the projection's rows."""
    B, T, Hq, Hkv, D = 2, 70, 4, 2, 64
    qkv = data(40, "bf16", B, T, Hq + 2 * Hkv, D).requires_grad_()
    env = dict(qkv=qkv, D=D, Hq=Hq, Hkv=Hkv)
    exec(readme("attention_ad("), env)
    do = data(41, "bf16", B, Hq, T, D)
    env["o"].backward(do)
    rows, table = qkv.detach().transpose(1, 2), fa.RotaryTable(D)
    q, k = fa.rotary(table, rows[:, :Hq], rows[:, Hq:Hq + Hkv])
    v = rows[:, Hq + Hkv:].contiguous()
    o, lse = fa.attention(q, k, v, causal=True)
    assert torch.equal(env["o"], o) and torch.equal(env["lse"], lse)
    dq, dk, dv = fa.attention_bwd(q, k, v, o, lse, do, causal=True)
    want = torch.cat((*fa.rotary(table, dq, dk, inverse=True), dv), 1).transpose(1, 2)
    assert torch.equal(qkv.grad, want)


def test_the_readme_s_serving_step(fa):  # noqa: F811
    """A prompt and single tokens over two layers, as it stands there, against attention over all rows at once."""
    B, Hq, Hkv, D, page, layers, total = 2, 4, 2, 64, 16, 2, 41
    pools = [[torch.zeros(B * 4, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(layers)]
    seq_len, next_pos = ints([0] * B), ints([0] * B)
    whole = [data(42 + i, "bf16", B, total, Hq + 2 * Hkv, D) for i in range(layers)]
    env = dict(caches=[fa.KVCache(*p, seq_len) for p in pools], Hq=Hq, Hkv=Hkv, table=fa.RotaryTable(D), seq_len=seq_len, next_pos=next_pos)
    out, at = [[] for _ in range(layers)], 0
    for T in (39, 1, 1):
        env.update(T=T, qkv=[x[:, at:at + T] for x in whole], o=[None] * layers, lse=[None] * layers)
        exec(readme("rotary_append("), env)
        for i in range(layers):
            out[i].append(env["o"][i])
        at += T
    assert seq_len.tolist() == next_pos.tolist() == [total] * B
    for i in range(layers):
        q, k, v = whole[i].transpose(1, 2).split([Hq, Hkv, Hkv], 1)
        q, k = fa.rotary(env["table"], q, k)
        want, _ = fa.attention(q, k, v.contiguous(), causal=True)
        # two kernels with sums in other orders: each within half a step of P's rounding, of |v| <= 5, and of its own
        assert (torch.cat(out[i], 2).double() - want.double()).abs().max() <= 5 * 2 * 2.0 ** -8 + 2 * 2.0 ** -8 * want.double().abs().max()
