"""The measured cases of attention's backward pass, of rotary positions, and of the cache's writes with the rotation
on the way.

Each case is one call that a training step or a serving loop makes for one layer.  ``run`` computes it in plain torch
operations (``own`` false) or through the package's entry points (``own`` true).

The formulas, for query head h and KV head c = h / (Hq / Hkv); J(i) are the keys that query i sees, off = Sk - Sq with the
bottom-right mask, 0 with the top-left one:

  backward  p_ij = exp(scale q_i.k_j - lse_i) for j in J(i), else 0;  delta_i = do_i.o_i - dlse_i
            ds_ij = p_ij (do_i.v_j - delta_i);  dq_i = scale sum_j ds_ij k_j;  dk_j = scale sum_hi ds_ij q_i;
            dv_j = sum_hi p_ij do_i   (sums over the query heads h of c and their rows i)
  rotary    pair p of a head turns by the angle t = position * frequency[p]:
            (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t);  inverse: by -t, which is its gradient too.
            The pair is elements p and p + rot / 2 (half layout) or 2p and 2p + 1 (interleaved) of the first rot elements
            of a head; the others pass as they are
  append    the queries, keys and values of token i < count[b], out of one projection's rows: queries and keys turn by
            position start[b] + i, keys and values also go to slot n_b + i of the cache, whose weight becomes 0
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- the cases

def listed():
    def bwd(name, B, heads, Sq, Sk, dtype, causal, std=1.0, dlse=False):
        return dict(name=name, op="backward", B=B, Hq=heads[0], Hkv=heads[1], D=heads[2], Sq=Sq, Sk=Sk, dtype=dtype, causal=causal, std=std, dlse=dlse)

    def rot(name, B, heads, T, dtype, turn, far, inverse):
        return dict(name=name, op="rotary", B=B, Hq=heads[0], Hkv=heads[1], D=heads[2], T=T, dtype=dtype, rot=turn[0], interleaved=turn[1],
                    scaling=turn[2], far=far, inverse=inverse)

    def app(name, B, heads, T, n, page, dtype, turn, ragged):
        return dict(name=name, op="append", B=B, Hq=heads[0], Hkv=heads[1], D=heads[2], T=T, n=n, page=page, dtype=dtype, rot=turn[0],
                    interleaved=turn[1], scaling=turn[2], ragged=ragged)

    return [
        # the smallest training step: two heads of one tile, all latency
        bwd("backward_small", 1, (2, 2, 64), 128, 128, "bf16", 1),
        # short sequences with small heads
        bwd("backward_short", 4, (16, 16, 64), 1024, 1024, "bf16", 1),
        # lengths that are no multiple of a tile, large logits, no mask, a loss that looks at lse too
        bwd("backward_odd_fp16", 8, (16, 16, 128), 2000, 2000, "fp16", 0, std=2.0, dlse=True),
        # a chunk of queries behind earlier keys, heads that share one in seven
        bwd("backward_chunk", 2, (14, 2, 128), 1000, 5000, "bf16", 2),
        # large heads
        bwd("backward_large_heads", 2, (32, 8, 256), 4096, 4096, "bf16", 1),
        # a long sequence: the most that a layer's backward pass computes
        bwd("backward_long", 1, (32, 8, 128), 16384, 16384, "bf16", 1),
        # one token of a few sequences far into their contexts: all latency
        rot("rotary_decode", 8, (32, 8, 128), 1, "bf16", (128, False, "none"), True, False),
        # a long prompt with frequencies stretched for it
        rot("rotary_prompt", 1, (32, 8, 128), 16384, "bf16", (128, False, "ramp"), False, False),
        # gradients back through the rotation of neighbours in half of each head, odd lengths
        rot("rotary_gradient", 3, (16, 16, 64), 1777, "fp16", (32, True, "linear"), False, True),
        # one new token of a batch
        app("append_decode", 16, (32, 8, 128), 1, 4096, 64, "bf16", (128, False, "none"), True),
        # chunks of prompts of mixed length, small pages, part of each head
        app("append_chunks", 8, (16, 16, 64), 500, 1500, 16, "fp16", (32, True, "linear"), True),
        # a whole prompt
        app("append_prompt", 1, (32, 8, 128), 16384, 0, 128, "bf16", (128, False, "ramp"), False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("backward", "backward", "rotary", "append"))
    Hq, Hkv, D = rng.choice(((32, 8, 128), (32, 8, 256), (16, 16, 64), (16, 16, 128), (24, 3, 128), (14, 2, 64), (6, 6, 256), (8, 1, 128), (2, 2, 64)))
    c = dict(op=op, B=log(1, 16), Hq=Hq, Hkv=Hkv, D=D, dtype=rng.choice(("bf16", "fp16")))
    if op == "backward":
        Sq = log(1, 16384)
        c.update(Sq=Sq, Sk=Sq if rng.random() < 0.6 else log(1, 16384), causal=rng.choice((0, 1, 1, 2)), std=rng.choice((1.0, 1.0, 2.0)),
                 dlse=rng.random() < 0.3)
        while c["B"] > 1 and c["B"] * Hq * c["Sq"] * c["Sk"] * D > 32 * 16384 ** 2 * 128 / 4:
            c["B"] -= 1
        while c["Hq"] * c["Sq"] * c["Sk"] * D > 32 * 16384 ** 2 * 128 / 4:
            c["Sq"], c["Sk"] = c["Sq"] // 2 + 1, c["Sk"] // 2 + 1
        return c
    c.update(rot=rng.choice((D, D, D // 2, D // 4)), interleaved=rng.random() < 0.4, scaling=rng.choice(("none", "linear", "ramp")), T=log(1, 16384))
    while c["B"] > 1 and c["B"] * c["T"] > 16384:
        c["B"] -= 1
    while c["B"] * c["T"] * (Hq + Hkv) * D > 16384 * 40 * 128:
        c["T"] -= c["T"] // 8
    if op == "rotary":
        c.update(far=rng.random() < 0.5, inverse=rng.random() < 0.5)
    else:
        c.update(n=log(1, 8192), page=rng.choice((16, 32, 48, 64, 128)), ragged=rng.random() < 0.7)
        while c["B"] * (c["n"] + c["T"]) > 131072:
            c["n"] //= 2
    return c


def _tokens(case):
    """(slots in the cache before the call, new tokens) of each sequence: part of the case, not of its values."""
    r = random.Random("%(n)d %(T)d %(B)d" % case)
    B, n, T = case["B"], case["n"], case["T"]
    if not case["ragged"]:
        return [n] * B, [T] * B
    return [n] + [r.randint(n // 2, n) for _ in range(B - 1)], [T] + [r.randint(max(1, T // 3), T) for _ in range(B - 1)]


def _pairs(Sq, Sk, causal):
    """Pairs of a query and a key that it sees."""
    if not causal:
        return Sq * Sk
    i = np.arange(Sq, dtype=np.int64) + 1 + (Sk - Sq if causal == 2 else 0)
    return int(np.clip(i, 0, Sk).sum())


def work(case):
    B, Hq, Hkv, D, op = (case[x] for x in ("B", "Hq", "Hkv", "D", "op"))
    row = 2 * D
    if op == "backward":
        q, k = B * Hq * case["Sq"], B * Hkv * case["Sk"]
        return {"bytes": 4 * q * row + 4 * k * row + q * (8 if case["dlse"] else 4), "flops": 10 * B * Hq * D * _pairs(case["Sq"], case["Sk"], case["causal"])}
    if op == "rotary":
        turned = B * case["T"] * (Hq + Hkv)
        return {"bytes": 2 * turned * row, "flops": 3 * turned * case["rot"]}
    new = sum(_tokens(case)[1])
    return {"bytes": new * (2 * (Hq + 2 * Hkv) * row + 2 * Hkv * row + 8 * Hkv), "flops": 3 * new * (Hq + Hkv) * case["rot"]}


# ---------------------------------------------------------------- inputs

def _frequencies(rot, scaling):
    """Radians a position, for each pair, and the amplitude: a base of 10000, as it is, or stretched for a longer context:
    every frequency by 4, or those of pairs that turn less than once in 4096 positions by 8, those that turn more than 32
    times not at all, and those between by a share that goes with the pair's number."""
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "ramp":
        at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        share = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f * (1 - share) + f / 8.0 * share, 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    B, Hq, Hkv, D, op = (case[x] for x in ("B", "Hq", "Hkv", "D", "op"))
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    normal = lambda *shape, std=1.0: (torch.randn(shape, generator=g, device=dev) * std).to(dt)  # noqa: E731
    if op == "backward":
        Sq, Sk, causal, std = case["Sq"], case["Sk"], case["causal"], case["std"]
        st = dict(op=op, scale=D ** -0.5, causal=causal, q=normal(B, Hq, Sq, D, std=std), k=normal(B, Hkv, Sk, D, std=std), v=normal(B, Hkv, Sk, D),
                  do=normal(B, Hq, Sq, D), dlse=torch.randn(B, Hq, Sq, generator=g, device=dev) if case["dlse"] else None)
        st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty(B, Hq, Sq, device=dev)
        for b, c, h in _groups(st):   # the forward pass, as it ran before
            s, shut = _scores(st, b, c, h)
            lse = torch.logsumexp(s, 3)
            st["lse"][b, h] = lse.reshape(-1, Sq)
            st["o"][b, h] = (s.sub_(lse[..., None]).exp_().masked_fill_(shut, 0.0) @ st["v"][b, c].float()[:, None]).reshape(-1, Sq, D).to(dt)
        return st
    f, amplitude = _frequencies(case["rot"], case["scaling"])
    st = dict(op=op, rot=case["rot"], interleaved=case["interleaved"], freq=torch.tensor(f, device=dev), amplitude=amplitude)
    if own:
        import programming_flashattention_fwd_gb300 as fa
        how = {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ramp": dict(scaling="ramp", factor=8.0, original=4096)}[case["scaling"]]
        st["table"] = fa.RotaryTable(D, rot=case["rot"], base=10000.0, interleaved=case["interleaved"], device=dev, **how)
    T = case["T"]
    heads = lambda x, lo, n: x.view(B, T, -1, D)[:, :, lo:lo + n].transpose(1, 2)  # noqa: E731
    if op == "rotary":
        start = r.integers(0, 131072 - T if case["far"] else 1, B)
        fused = normal(B, T, (Hq + 2 * Hkv) * D)
        st.update(start=ints(start), inverse=case["inverse"], fused=fused)
        if case["inverse"]:   # gradients of the rotated tensors, to the gradients of the projection's rows
            st.update(q=normal(B, Hq, T, D), k=normal(B, Hkv, T, D), q_out=heads(fused, 0, Hq), k_out=heads(fused, Hq, Hkv))
        else:
            st.update(q=heads(fused, 0, Hq), k=heads(fused, Hq, Hkv), q_out=torch.zeros(B, Hq, T, D, dtype=dt, device=dev),
                      k_out=torch.zeros(B, Hkv, T, D, dtype=dt, device=dev))
        return st
    lens, new = _tokens(case)
    page = case["page"]
    per = (max(n + t for n, t in zip(lens, new)) + page - 1) // page
    pool = B * per + 3                      # a few pages belong to nobody
    fused = normal(B, T, (Hq + 2 * Hkv) * D)
    st.update(k_pool=normal(pool, Hkv, page, D), v_pool=normal(pool, Hkv, page, D), table_=ints(r.permutation(pool)[:B * per].reshape(B, per)),
              seq_len=ints(lens), count=ints(new), start=ints([n + 7 * b for b, n in enumerate(lens)]),
              q=heads(fused, 0, Hq), k=heads(fused, Hq, Hkv), v=heads(fused, Hq + Hkv, Hkv),
              weight=torch.rand(B, Hkv, per * page, generator=g, device=dev), pos=torch.zeros(B, Hkv, per * page, dtype=torch.int32, device=dev))
    for x in "qkv":
        st[x + "_out"] = torch.zeros(st[x].shape, dtype=dt, device=dev)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        import programming_flashattention_fwd_gb300 as fa
        if st["op"] == "backward":
            dq, dk, dv = fa.attention_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], causal=st["causal"], scale=st["scale"], dlse=st["dlse"])
            return {"dq": dq, "dk": dk, "dv": dv}
        if st["op"] == "rotary":
            fa.rotary(st["table"], st["q"], st["k"], start=st["start"], inverse=st["inverse"], q_out=st["q_out"], k_out=st["k_out"])
            return {"fused": st["fused"]} if st["inverse"] else {"q": st["q_out"], "k": st["k_out"]}
        cache = fa.KVCache(st["k_pool"], st["v_pool"], st["seq_len"], st["table_"])
        q, k, v = fa.rotary_append(cache, st["table"], st["q"], st["k"], st["v"], start=st["start"], count=st["count"], weight=st["weight"], pos=st["pos"],
                                   q_out=st["q_out"], k_out=st["k_out"], v_out=st["v_out"])
        return {"q": q, "k": k, "v": v, "k_pool": st["k_pool"], "v_pool": st["v_pool"], "weight": st["weight"], "pos": st["pos"]}
    return {"backward": _backward, "rotary": _rotary, "append": _append}[st["op"]](st)


def _groups(st):
    """(sequence, KV heads, their query heads): as many KV heads at a time as keep a product of scores within 2^30 values."""
    B, Hq, Sq, _ = st["q"].shape
    Hkv, Sk = st["k"].shape[1:3]
    group = Hq // Hkv
    n = max(1, 2 ** 30 // max(group * Sq * Sk, 1))
    for b in range(B):
        for c in range(0, Hkv, n):
            e = min(c + n, Hkv)
            yield b, slice(c, e), slice(c * group, e * group)


def _shut(st, Sq, Sk):
    """Pairs that the mask shuts, [Sq, Sk]."""
    i, j = torch.arange(Sq, device=st["q"].device)[:, None], torch.arange(Sk, device=st["q"].device)
    return j > i + (Sk - Sq if st["causal"] == 2 else 0) if st["causal"] else torch.zeros(Sq, Sk, dtype=torch.bool, device=st["q"].device)


def _scores(st, b, c, h):
    """Masked scores [KV heads, group, Sq, Sk] and the mask."""
    k = st["k"][b, c].float()
    q = st["q"][b, h].float().reshape(k.shape[0], -1, *st["q"].shape[2:])
    shut = _shut(st, q.shape[2], k.shape[1])
    return (q @ k.transpose(1, 2)[:, None]).mul_(st["scale"]).masked_fill_(shut, -float("inf")), shut


def _backward(st):
    dq, dk, dv = torch.empty_like(st["q"]), torch.empty_like(st["k"]), torch.empty_like(st["v"])
    delta = (st["do"].float() * st["o"].float()).sum(3)
    if st["dlse"] is not None:
        delta -= st["dlse"]
    for b, c, h in _groups(st):
        p, shut = _scores(st, b, c, h)
        n, group, Sq, _ = p.shape
        rows = lambda x: x[b, h].float().reshape(n, group * Sq, *x.shape[3:])  # noqa: E731
        p = p.reshape(n, group * Sq, -1).sub_(rows(st["lse"])[..., None]).exp_()
        p.view(n, group, Sq, -1).masked_fill_(shut, 0.0)
        do, k, v = rows(st["do"]), st["k"][b, c].float(), st["v"][b, c].float()
        dv[b, c] = (p.transpose(1, 2) @ do).to(dv.dtype)
        ds = (do @ v.transpose(1, 2)).sub_(rows(delta)[..., None]).mul_(p).mul_(st["scale"])
        dk[b, c] = (ds.transpose(1, 2) @ rows(st["q"])).to(dk.dtype)
        dq[b, h] = (ds @ k).reshape(n * group, Sq, -1).to(dq.dtype)
    return {"dq": dq, "dk": dk, "dv": dv}


def _turn(st, x, position, back=False):
    """x [B, H, T, D] turned by position [B, T]; angles in 64 bits."""
    rot = st["rot"]
    angle = (position.double()[..., None] * st["freq"])[:, None]
    cos, sin = (angle.cos() * st["amplitude"]).float(), (angle.sin() * st["amplitude"]).float()
    if back:
        sin = -sin
    y = x.float().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if st["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., a].float(), x[..., b].float()
    y[..., a], y[..., b] = u * cos - v * sin, u * sin + v * cos
    return y.to(x.dtype)


def _rotary(st):
    position = st["start"].long()[:, None] + torch.arange(st["q"].shape[2], device=st["q"].device)
    for x in "qk":
        st[x + "_out"].copy_(_turn(st, st[x], position, st["inverse"]))
    return {"fused": st["fused"]} if st["inverse"] else {"q": st["q_out"], "k": st["k_out"]}


def _append(st):
    T, page = st["q"].shape[2], st["k_pool"].shape[2]
    position = st["start"].long()[:, None] + torch.arange(T, device=st["q"].device)
    here = torch.arange(T, device=st["q"].device) < st["count"][:, None]
    q, k, v = _turn(st, st["q"], position), _turn(st, st["k"], position), st["v"]
    for out, x in ((st["q_out"], q), (st["k_out"], k), (st["v_out"], v)):
        out.copy_(torch.where(here[:, None, :, None], x, out))
    b, i = torch.nonzero(here, as_tuple=True)
    slot = st["seq_len"].long()[b] + i
    at, row = st["table_"][b, slot // page].long(), slot % page
    st["k_pool"][at, :, row] = k[b, :, i]
    st["v_pool"][at, :, row] = v[b, :, i]
    st["weight"][b, :, slot] = 0.0
    st["pos"][b, :, slot] = position[b, i].to(torch.int32)[:, None]
    return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"], "weight": st["weight"], "pos": st["pos"]}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    def backward(st):
        q, k, v, do = (st[x].double() for x in ("q", "k", "v", "do"))
        B, Hq, Sq, D = q.shape
        Hkv, Sk = k.shape[1:3]
        off = {0: Sk, 1: 0, 2: Sk - Sq}[st["causal"]]
        delta = torch.einsum("bhid,bhid->bhi", do, st["o"].double())
        if st["dlse"] is not None:
            delta = delta - st["dlse"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b in range(B):
            for h in range(Hq):
                c = h * Hkv // Hq
                for lo in range(0, Sq, 2048):
                    hi = min(lo + 2048, Sq)
                    n = max(0, min(Sk, hi + off))   # no row of these sees a key behind
                    if n == 0:
                        continue
                    x, y = q[b, h, lo:hi], do[b, h, lo:hi]
                    p = torch.exp(torch.addmm(-st["lse"][b, h, lo:hi, None].double(), x, k[b, c, :n].T, alpha=st["scale"]))
                    p = torch.where(torch.ones_like(p, dtype=torch.bool).tril(lo + off), p, 0.0)
                    e = p * (y @ v[b, c, :n].T - delta[b, h, lo:hi, None]) * st["scale"]
                    dq[b, h, lo:hi] = e @ k[b, c, :n]
                    dk[b, c, :n] += e.T @ x
                    dv[b, c, :n] += p.T @ y
        return {"dq": dq, "dk": dk, "dv": dv}

    def turned(st, x, start, sign):
        """Complex multiplication by amplitude e^(i angle)."""
        rot, T = st["rot"], x.shape[2]
        x = x.double().clone(memory_format=torch.contiguous_format)
        where = torch.arange(rot, device=x.device)
        where = where.view(-1, 2) if st["interleaved"] else where.view(2, -1).T
        z = torch.complex(x[..., where[:, 0]], x[..., where[:, 1]])
        t = start.double()[:, None] + torch.arange(T, device=x.device, dtype=torch.float64)
        z = z * torch.polar(torch.full_like(t, st["amplitude"])[..., None].expand(*t.shape, rot // 2).contiguous(), sign * t[..., None] * st["freq"])[:, None]
        x[..., where[:, 0]], x[..., where[:, 1]] = z.real, z.imag
        return x

    def rotary(st):
        q, k = (turned(st, st[x], st["start"], -1.0 if st["inverse"] else 1.0) for x in "qk")
        if not st["inverse"]:
            return {"q": q, "k": k}
        whole = st["fused"].double()
        Hq, Hkv, D = q.shape[1], k.shape[1], q.shape[3]
        whole[..., :Hq * D] = q.transpose(1, 2).flatten(2)
        whole[..., Hq * D:(Hq + Hkv) * D] = k.transpose(1, 2).flatten(2)
        return {"fused": whole}

    def append(st):
        q, k, v = turned(st, st["q"], st["start"], 1.0), turned(st, st["k"], st["start"], 1.0), st["v"].double()
        out = [st[x + "_out"].double() for x in "qkv"]
        pools = [st["k_pool"].double(), st["v_pool"].double()]
        weight, pos, page = st["weight"].double(), st["pos"].cpu().numpy(), st["k_pool"].shape[2]
        table = st["table_"].cpu().numpy()
        for b in range(len(table)):
            n, t, at = int(st["seq_len"][b]), int(st["count"][b]), int(st["start"][b])
            for y, x in zip(out, (q, k, v)):
                y[b, :, :t] = x[b, :, :t]
            slot = np.arange(n, n + t)
            pages, rows = (torch.tensor(x).long().to(q.device) for x in (table[b, slot // page], slot % page))
            for y, x in zip(pools, (k, v)):
                y[pages, :, rows] = x[b, :, :t].transpose(0, 1)
            weight[b, :, n:n + t] = 0.0
            pos[b, :, n:n + t] = np.arange(at, at + t)
        return {"q": out[0], "k": out[1], "v": out[2], "k_pool": pools[0], "v_pool": pools[1], "weight": weight, "pos": pos}

    st = prepare(case, seed)
    return {"backward": backward, "rotary": rotary, "append": append}[st["op"]](st)
