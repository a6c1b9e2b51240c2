"""The cache operators' measured cases: attention for drafted tokens over a paged key/value cache, the
cache's writes, the accumulated attention weight of its slots, and eviction by that weight.

Each case is one call that a serving loop makes for one layer.  ``run`` computes it in plain torch
operations (``own`` false) or through the package's entry points (``own`` true).

The formulas, for sequence b, query head h and KV head c = h / (Hq / Hkv); the cache holds n_b slots
of b, slot s on row s % page of page table[b, s / page]:

  attend    o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i.k_j - lse_i), over the n_b slots and the drafted
            tokens j on the path from i to its root (i itself included); lse_i = ln sum_j exp(scale q_i.k_j)
  append    slot n_b + i takes the key and value of drafted token path[b, i], i < count[b]
  weigh     out[b, c, s] = weight[b, c, s] + sum over the heads of c and the rows i < count[b] with
            s < n_b - count[b] + i + 1 of exp(scale q_i.k_s - lse_i)
  evict     of n_b slots keep those of the first and last positions and, by weight, others, `keep` in
            all (ties: the lowest slot); kept slots at keep or above move, in order, to the free slots below
"""
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- the cases

def listed():
    def case(name, op, heads, n, T, page, dtype, B, **more):
        return dict(name=name, op=op, B=B, Hq=heads[0], Hkv=heads[1], D=heads[2], n=n, T=T, page=page, dtype=dtype, **more)

    return [
        # one new token of one sequence: the smallest step of a decoding loop, all latency
        case("attend_one_token", "attend", (32, 8, 128), 4096, 1, 64, "bf16", 1, ragged=False),
        # a batch of sequences of mixed length with small trees, small pages, no shared heads
        case("attend_ragged_trees", "attend", (16, 16, 128), 2000, 24, 16, "fp16", 8, ragged=True),
        # long contexts with wide trees: the most that a drafting step reads
        case("attend_long_wide", "attend", (32, 8, 128), 16384, 64, 128, "bf16", 8, ragged=True),
        # large heads, an odd tree
        case("attend_large_heads", "attend", (32, 8, 256), 4096, 17, 32, "bf16", 4, ragged=True),
        # the accepted tokens' weights on long caches, after a drafting step
        case("weigh_accepted", "weigh", (32, 8, 128), 16384, 64, 128, "bf16", 8, ragged=True, prompt=False),
        # a long prompt's weights: every query against every earlier key
        case("weigh_long_prompt", "weigh", (32, 8, 128), 16384, 16384, 128, "bf16", 1, ragged=False, prompt=True),
        # short prompts of mixed length with small heads
        case("weigh_short_prompts", "weigh", (16, 16, 64), 1024, 1024, 64, "fp16", 4, ragged=True, prompt=True),
        # the accepted tokens of a drafting step
        case("append_accepted", "append", (32, 8, 128), 4096, 24, 64, "bf16", 8, ragged=True, prompt=False),
        # a whole prompt
        case("append_prompt", "append", (32, 8, 128), 16384, 16384, 128, "bf16", 1, ragged=False, prompt=True),
        # a decoding loop that has grown past its budget by a few steps
        case("evict_few", "evict", (32, 8, 128), 4160, 0, 64, "bf16", 8, ragged=False, keep=4096),
        # a long prompt cut to its budget
        case("evict_long_prompt", "evict", (32, 8, 128), 16384, 0, 128, "bf16", 4, ragged=False, keep=2048),
        # mixed lengths, small heads, an odd budget
        case("evict_ragged", "evict", (16, 16, 64), 2000, 0, 16, "fp16", 16, ragged=True, keep=777),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("attend", "weigh", "append", "evict"))
    Hq, Hkv, D = rng.choice(((32, 8, 128), (32, 8, 256), (16, 16, 64), (16, 16, 128), (24, 3, 128), (14, 2, 64), (6, 6, 256)))
    c = dict(op=op, B=log(1, 16), Hq=Hq, Hkv=Hkv, D=D, n=log(60, 16384), T=0, page=rng.choice((16, 32, 48, 64, 128)),
             dtype=rng.choice(("bf16", "fp16")), ragged=rng.random() < 0.7)
    most = 8 * 16384 * 1024
    if op in ("weigh", "append"):
        c["prompt"] = rng.random() < 0.5
    if op == "attend" or not c.get("prompt", True):
        c["T"] = log(1, 64)
    if op == "evict":
        c["keep"] = max(1, int(c["n"] * rng.choice((0.1, 0.35, 0.6, 0.97))))
    if c.get("prompt"):
        c["T"] = c["n"]
        while op == "weigh" and c["B"] > 1 and c["B"] * c["Hq"] * c["n"] ** 2 * D > 32 * 16384 ** 2 * 128 / 2:
            c["B"] -= 1
        c["Hq"], c["Hkv"] = (Hq, Hkv) if c["n"] * c["n"] * c["B"] * Hq * D <= 32 * 16384 ** 2 * 128 else (16, 4)
        most = 16384 * 1024 if op == "append" else most
    while c["B"] > 1 and c["B"] * c["n"] * Hkv * D > most:
        c["B"] -= 1
    if c["n"] * Hkv * D > most:
        c["n"] = most // (Hkv * D)
        c["T"] = min(c["T"], c["n"])
    return c


def _lengths(case):
    """(slots in the cache before the call, new tokens) of each sequence: part of the case, not of its values."""
    r = random.Random("%(op)s %(n)d %(T)d %(B)d" % case)
    B, n, T = case["B"], case["n"], case["T"]
    pick = (lambda lo, hi: r.randint(lo, hi)) if case["ragged"] else (lambda lo, hi: hi)
    first = lambda lo, hi: [hi] + [pick(lo, hi) for _ in range(B - 1)]  # noqa: E731
    if case["op"] == "evict":
        return first(n // 2, n), [0] * B
    if case.get("prompt"):
        new = first(max(1, n // 3), T)
        return ([0] * B if case["op"] == "append" else list(new)), new
    if case["op"] == "attend":
        return first(n // 2, n), first(max(1, T // 2), T)
    few = min(T, 6)   # accepted tokens
    return first(max(few, n // 2), max(few, n)), [r.randint(1, few) for _ in range(B)]


def work(case):
    lens, new = _lengths(case)
    Hq, Hkv, D, op = case["Hq"], case["Hkv"], case["D"], case["op"]
    row = 2 * D
    if op == "attend":
        pairs = sum(t * n + t * (t + 1) / 2 for n, t in zip(lens, new))
        rows = sum(new)
        nbytes = 2 * row * Hkv * (sum(lens) + rows) + rows * (Hq * (2 * row + 4) + 4)
        return {"bytes": nbytes, "flops": 4 * Hq * D * pairs}
    if op == "append":
        return {"bytes": 4 * row * Hkv * sum(new) + 8 * Hkv * sum(new), "flops": 0}
    if op == "weigh":
        pairs = sum(t * (n - t) + t * (t + 1) / 2 for n, t in zip(lens, new))
        nbytes = sum(Hkv * n * (row + 8) + Hq * t * (row + 4) for n, t in zip(lens, new))
        return {"bytes": nbytes, "flops": 2 * Hq * D * pairs}
    # evict: weights and positions are read and the kept ones written; how many rows move depends on
    # the weights, and is taken as the expected share of the slots at `keep` or above
    nbytes = 0
    for n in lens:
        k = min(n, case["keep"])
        moved = (n - k) * k / max(n, 1)
        nbytes += Hkv * (8 * (n + k) + 4 * row * moved)
    return {"bytes": nbytes, "flops": 0}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    def tree(r, T, t_b):
        """Parents of a drafted tree: a token follows one of the last few before it, or starts a branch."""
        parent = np.full(T, -1, np.int32)
        for t in range(1, t_b):
            parent[t] = t - 1 - min(t - 1, int(r.exponential(2.0))) if r.random() < 0.95 else -1
        seen = np.zeros((T, T), bool)
        for t in range(t_b):
            if parent[t] >= 0:
                seen[t] = seen[parent[t]]
            seen[t, t] = True
        return parent, seen

    def rows_of(cache, table, n):
        """The first n slots of a sequence as float32 [Hkv, n, D]."""
        page = cache.shape[2]
        x = cache[table[:(n + page - 1) // page].long()].transpose(0, 1)
        return x.reshape(x.shape[0], -1, x.shape[3])[:, :n].float()

    def lse_of_cache(st, q, lens, new, path):
        """lse of the query rows over the slots they see, as the attention that ran before would have left it."""
        B, Hq, T, D = q.shape
        lse = torch.full((B, Hq, T), -float("inf"), device=q.device)
        for b, (n, t) in enumerate(zip(lens, new)):
            k = rows_of(st["k"], st["table"][b], n)
            rows = torch.arange(t, device=q.device) if path is None else path[b, :t].long()
            for h in range(Hq):
                s = (q[b, h, rows].float() @ k[h // (Hq // k.shape[0])].T) * st["scale"]
                seen = torch.arange(n, device=q.device)[None, :] < (n - t + 1 + torch.arange(t, device=q.device))[:, None]
                lse[b, h, rows] = torch.logsumexp(s.masked_fill(~seen, -float("inf")), 1)
        return lse

    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    B, Hq, Hkv, D, T, page, op = (case[x] for x in ("B", "Hq", "Hkv", "D", "T", "page", "op"))
    lens, new = _lengths(case)
    per = (max(n + (t if op == "append" else 0) for n, t in zip(lens, new)) + page - 1) // page
    pool = B * per + 3                      # a few pages belong to nobody
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev).to(dt)  # noqa: E731
    st = dict(op=op, scale=D ** -0.5, k=normal(pool, Hkv, page, D), v=normal(pool, Hkv, page, D),
              table=ints(r.permutation(pool)[:B * per].reshape(B, per)), seq_len=ints(lens))
    slots = per * page
    if op == "attend":
        trees = [tree(r, T, t) for t in new]
        st.update(q=normal(B, Hq, T, D), k_new=normal(B, Hkv, T, D), v_new=normal(B, Hkv, T, D), parent=ints([p for p, _ in trees]),
                  seen=torch.tensor(np.stack([s for _, s in trees]), device=dev), draft_len=ints(new))
        st.update(o=torch.zeros_like(st["q"]), lse=torch.zeros(B, Hq, T, device=dev))
        return st
    weight = torch.empty(B, Hkv, slots, device=dev).exponential_(1.0, generator=g)
    if op == "evict":
        # positions in an order that earlier evictions have left; heavy-tailed weights, and some slots that nothing looked at
        pos = np.stack([np.stack([r.permutation(slots) for _ in range(Hkv)]) for _ in range(B)])
        weight = weight ** 3 * (torch.rand(weight.shape, generator=g, device=dev) > 0.02)
        st.update(weight=weight, pos=ints(pos), next_pos=ints([slots] * B), keep=case["keep"], first=min(4, case["keep"] // 4),
                  last=min(32, case["keep"] // 4), weight_out=torch.zeros_like(weight), pos_out=torch.zeros(B, Hkv, slots, dtype=torch.int32, device=dev))
        return st
    path = None
    if not case["prompt"]:
        path = np.full((B, T), -1, np.int32)
        for b, t in enumerate(new):
            path[b, :t] = np.sort(r.choice(T, t, replace=False))
        path = ints(path)
    st.update(path=path, count=ints(new), weight=weight)
    if op == "append":
        st.update(k_new=normal(B, Hkv, T, D), v_new=normal(B, Hkv, T, D), pos=torch.zeros(B, Hkv, slots, dtype=torch.int32, device=dev),
                  start=ints([n + 5 for n in lens]))
    else:
        st["q"] = normal(B, Hq, T, D)
        st.update(lse=lse_of_cache(st, st["q"], lens, new, path), out=torch.zeros_like(weight))
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        import programming_flashattention_fwd_gb300 as fa
        cache = fa.KVCache(st["k"], st["v"], st["seq_len"], st["table"])
        if st["op"] == "attend":
            o, lse = fa.tree_attention(st["q"], st["k_new"], st["v_new"], cache, parent=st["parent"], draft_len=st["draft_len"], scale=st["scale"],
                                       o=st["o"], lse=st["lse"])
            return {"o": o, "lse": lse}
        if st["op"] == "append":
            fa.cache_append(cache, st["k_new"], st["v_new"], path=st["path"], count=st["count"], weight=st["weight"], pos=st["pos"], start=st["start"])
            return {"k": st["k"], "v": st["v"], "weight": st["weight"], "pos": st["pos"]}
        if st["op"] == "weigh":
            return {"weight": fa.cache_weights(cache, st["q"], st["lse"], st["weight"], path=st["path"], count=st["count"], scale=st["scale"], out=st["out"])}
        new_len = fa.cache_evict(cache, st["weight"], st["pos"], st["keep"], first=st["first"], last=st["last"], next_pos=st["next_pos"],
                                 weight_out=st["weight_out"], pos_out=st["pos_out"])
        return {"len": new_len, "k": st["k"], "v": st["v"], "weight": st["weight_out"], "pos": st["pos_out"]}
    return {"attend": _attend, "append": _append, "weigh": _weigh, "evict": _evict}[st["op"]](st)


def _dense(cache, table):
    """Every slot of every sequence as float32 [B, Hkv, slots, D]."""
    x = cache[table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4]).float()


def _attend(st):
    q, lens = st["q"], st["seq_len"].long()
    B, Hq, T, D = q.shape
    Hkv = st["k"].shape[1]
    rows = q.float().reshape(B, Hkv, -1, D) * st["scale"]
    k, v = _dense(st["k"], st["table"]), _dense(st["v"], st["table"])
    here = torch.arange(k.shape[2], device=q.device) < lens[:, None]
    v = torch.where(here[:, None, :, None], v, 0.0)
    old = (rows @ k.transpose(2, 3)).masked_fill_(~here[:, None, None, :], -float("inf"))
    new = (rows @ st["k_new"].float().transpose(2, 3)).reshape(B, Hq, T, T).masked_fill(~st["seen"][:, None], -float("inf")).reshape(B, Hkv, -1, T)
    top = torch.maximum(old.amax(3) if old.shape[3] else -float("inf"), new.amax(3))
    top = torch.where(torch.isinf(top), 0.0, top)[..., None]
    old, new = old.sub_(top).exp_(), (new - top).exp()
    total = old.sum(3) + new.sum(3)
    o = (old @ v + new @ st["v_new"].float()) / torch.where(total > 0, total, 1.0)[..., None]
    lse = total.log() + top[..., 0]
    valid = torch.arange(T, device=q.device)[None, :] < st["draft_len"][:, None]
    st["o"].copy_(torch.where(valid[:, None, :, None], o.reshape(q.shape).to(q.dtype), st["o"]))
    st["lse"].copy_(torch.where(valid[:, None, :], lse.reshape(B, Hq, T), st["lse"]))
    return {"o": st["o"], "lse": st["lse"]}


def _append(st):
    T, page = st["k_new"].shape[2], st["k"].shape[2]
    b, i = torch.nonzero(torch.arange(T, device=st["k"].device)[None, :] < st["count"][:, None], as_tuple=True)
    src = i if st["path"] is None else st["path"][b, i].long()
    slot = st["seq_len"].long()[b] + i
    at, row = st["table"][b, slot // page].long(), slot % page
    st["k"][at, :, row] = st["k_new"][b, :, src]
    st["v"][at, :, row] = st["v_new"][b, :, src]
    st["weight"][b, :, slot] = 0.0
    st["pos"][b, :, slot] = (st["start"][b] + i).to(torch.int32)[:, None]
    return {"k": st["k"], "v": st["v"], "weight": st["weight"], "pos": st["pos"]}


def _weigh(st):
    q, n, t = st["q"], st["seq_len"].long(), st["count"].long()
    B, Hq, T, D = q.shape
    k = _dense(st["k"], st["table"])
    Hkv = k.shape[1]
    i = torch.arange(T, device=q.device).expand(B, T)
    if st["path"] is not None:   # the accepted rows, in the order of their slots
        src = st["path"].long().clamp_min(0)[:, None, :].expand(B, Hq, T)
        q, lse = q.gather(2, src[..., None].expand(q.shape)), st["lse"].gather(2, src)
    else:
        lse = st["lse"]
    sees = torch.where(i < t[:, None], n[:, None] - t[:, None] + i + 1, 0)                    # slots that row i sees
    p = q.float().reshape(B, Hkv, -1, D).mul_(st["scale"]) @ k.transpose(2, 3)
    p = p.sub_(lse.reshape(B, Hkv, -1, 1)).exp_().reshape(B, Hkv, Hq // Hkv, T, -1)
    p.masked_fill_((torch.arange(p.shape[4], device=q.device) >= sees[..., None])[:, None, None], 0.0)
    here = torch.arange(p.shape[4], device=q.device) < n[:, None]
    st["out"].copy_(torch.where(here[:, None], st["weight"] + p.sum((2, 3)), st["out"]))
    return {"weight": st["out"]}


def _evict(st):
    w, pos, n, m, page = st["weight"], st["pos"], st["seq_len"].long(), st["keep"], st["k"].shape[2]
    slot = torch.arange(w.shape[2], device=w.device)
    here = (slot < n[:, None])[:, None]
    safe = (pos < st["first"]) | (pos >= (st["next_pos"] - st["last"])[:, None, None])
    rank = torch.where(safe, torch.inf, w).masked_fill(~here, -1.0).sort(dim=2, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter_(2, rank[..., :m], True) & here
    b, h, dst = torch.nonzero(here & ~kept & (slot < m) & (n[:, None, None] > m), as_tuple=True)
    src = torch.nonzero(kept & (slot >= m))[:, 2]
    for_ = lambda s: (st["table"][b, s // page].long(), h, s % page)  # noqa: E731
    st["k"][for_(dst)] = st["k"][for_(src)]
    st["v"][for_(dst)] = st["v"][for_(src)]
    left = torch.clamp(n, max=m)
    stay = (slot < left[:, None])[:, None]
    st["weight_out"].copy_(torch.where(stay, w, st["weight_out"]))
    st["pos_out"].copy_(torch.where(stay, pos, st["pos_out"]))
    st["weight_out"][b, h, dst] = w[b, h, src]
    st["pos_out"][b, h, dst] = pos[b, h, src]
    return {"len": left.to(torch.int32), "k": st["k"], "v": st["v"], "weight": st["weight_out"], "pos": st["pos_out"]}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    def slots(st, which, b, head, n):
        page = st["k"].shape[2]
        return torch.cat([st[which][int(p), head] for p in st["table"][b, :(n + page - 1) // page].tolist()] + [st[which][:0, 0, 0]])[:n].double()

    def attend(st):
        q = st["q"].double()
        B, Hq, T, D = q.shape
        group = Hq // st["k"].shape[1]
        o, lse = st["o"].double(), st["lse"].double()
        for b in range(B):
            n, t = int(st["seq_len"][b]), int(st["draft_len"][b])
            parent = st["parent"][b].tolist()
            open_ = torch.zeros(t, n + t, dtype=torch.bool)
            open_[:, :n] = True
            for i in range(t):
                j = i
                while j >= 0:
                    open_[i, n + j] = True
                    j = parent[j]
            shut = (~open_).to(q.device)
            for h in range(Hq):
                k = torch.cat([slots(st, "k", b, h // group, n), st["k_new"][b, h // group, :t].double()])
                v = torch.cat([slots(st, "v", b, h // group, n), st["v_new"][b, h // group, :t].double()])
                s = (q[b, h, :t] @ k.T * st["scale"]).masked_fill(shut, -float("inf"))
                lse[b, h, :t] = torch.logsumexp(s, 1)
                o[b, h, :t] = torch.softmax(s, 1) @ v
        return {"o": o, "lse": lse}

    def append(st):
        k, v, weight, pos = st["k"].double(), st["v"].double(), st["weight"].double(), st["pos"].cpu().numpy()
        page = st["k"].shape[2]
        table, path = st["table"].cpu().numpy(), None if st["path"] is None else st["path"].cpu().numpy()
        for b in range(len(table)):
            n, t = int(st["seq_len"][b]), int(st["count"][b])
            s = np.arange(n, n + t)
            at, row = torch.tensor(table[b, s // page]).long().to(k.device), torch.tensor(s % page).to(k.device)
            src = torch.tensor(np.arange(t) if path is None else path[b, :t]).long().to(k.device)
            k[at, :, row] = st["k_new"][b][:, src].transpose(0, 1).double()
            v[at, :, row] = st["v_new"][b][:, src].transpose(0, 1).double()
            weight[b, :, n:n + t] = 0
            pos[b, :, n:n + t] = int(st["start"][b]) + np.arange(t)
        return {"k": k, "v": v, "weight": weight, "pos": pos}

    def weigh(st):
        q, lse, out = st["q"], st["lse"].double(), st["out"].double()
        B, Hq, T, D = q.shape
        group = Hq // st["k"].shape[1]
        for b in range(B):
            n, t = int(st["seq_len"][b]), int(st["count"][b])
            rows = torch.arange(t, device=q.device) if st["path"] is None else st["path"][b, :t].long()
            for c in range(Hq // group):
                k = slots(st, "k", b, c, n)
                out[b, c, :n] = st["weight"][b, c, :n].double()
                for h in range(c * group, (c + 1) * group):
                    for i in range(0, t, 2048):   # rows i .. i + 2047 see the slots below n - t + i + 2048
                        at = rows[i:i + 2048]
                        top = min(n, n - t + i + len(at))
                        p = torch.exp(q[b, h, at].double() @ k[:top].T * st["scale"] - lse[b, h, at, None])
                        out[b, c, :top] += p.tril(n - t + i).sum(0)
        return {"weight": out}

    def evict(st):
        k, v, w, pos = st["k"].double(), st["v"].double(), st["weight"].cpu().numpy(), st["pos"].cpu().numpy()
        wo, po, table = st["weight_out"].cpu().numpy().astype(np.float64), st["pos_out"].cpu().numpy(), st["table"].cpu().numpy()
        page, left = st["k"].shape[2], []
        for b in range(len(w)):
            n, m = int(st["seq_len"][b]), st["keep"]
            left.append(min(n, m))
            for h in range(w.shape[1]):
                weights, where = w[b, h, :n].copy(), pos[b, h, :n].copy()
                safe = (where < st["first"]) | (where >= int(st["next_pos"][b]) - st["last"])
                kept = np.sort(np.lexsort((np.arange(n), -weights.astype(np.float64), ~safe))[:m])
                dst, src = np.setdiff1d(np.arange(min(n, m)), kept), kept[kept >= m]
                here, there = ((torch.tensor(table[b, s // page]).long().to(k.device), torch.tensor(s % page).to(k.device)) for s in (dst, src))
                for x in (k, v):
                    x[here[0], h, here[1]] = x[there[0], h, there[1]]
                weights[dst], where[dst] = weights[src], where[src]
                wo[b, h, :min(n, m)], po[b, h, :min(n, m)] = weights[:min(n, m)], where[:min(n, m)]
        return {"len": np.asarray(left, np.int32), "k": k, "v": v, "weight": wo, "pos": po}

    st = prepare(case, seed)
    return {"attend": attend, "append": append, "weigh": weigh, "evict": evict}[st["op"]](st)
