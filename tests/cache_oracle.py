"""The cache operators in float64 numpy, from their definitions in include/fa.h: the oracle of the
cache tests.  Shares no code with the library."""
import numpy as np


def path_of(parent, t):
    """The drafted tokens that token t sees, from itself to its root."""
    out = [t]
    while True:
        up = int(parent[out[-1]])
        if not 0 <= up < out[-1]:
            return out
        out.append(up)


def slots_of(pool, table, n):
    """The first n slots of a sequence: [Hkv, n, D] float64 (pool [num_pages, Hkv, page, D])."""
    page = pool.shape[2]
    rows = [pool[table[s // page], :, s % page] for s in range(n)]
    return np.stack(rows, 1) if rows else np.zeros((pool.shape[1], 0, pool.shape[3]))


def attend(q, k_new, v_new, k, v, table, seq_len, parent, draft_len, scale):
    """o, lse and the bound's ingredients: pv = sum_j p_j |v_j|, av = sum_j |v_j|, qk = max_j scale sum |q||k|."""
    B, Hq, T, D = q.shape
    group = Hq // k_new.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    pv, av, qk = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        n, t = int(seq_len[b]), T if draft_len is None else int(draft_len[b])
        kc, vc = slots_of(k, table[b], n), slots_of(v, table[b], n)
        for i in range(t):
            seen = path_of(parent[b], i) if parent is not None else list(range(i + 1))
            for h in range(Hq):
                c = h // group
                kk = np.concatenate([kc[c], k_new[b, c, seen]])
                vv = np.concatenate([vc[c], v_new[b, c, seen]])
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (kk @ q[b, h, i])
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    lse[b, h, i] = m + np.log(total)
                    p /= total
                    o[b, h, i] = p @ vv
                    pv[b, h, i] = p @ np.abs(vv)
                    av[b, h, i] = np.abs(vv).sum(0)
                    qk[b, h, i] = scale * (np.abs(kk) @ np.abs(q[b, h, i])).max()
    return o, lse, pv, av, qk


def weigh(q, lse, k, table, seq_len, path, count, causal, scale, group):
    """sum over rows and heads of exp(scale q.k - lse): [B, Hkv, slots in use] as a list per sequence, with
    the largest scale sum |q||k| and |lse| among the rows that count."""
    B, Hq, T, D = q.shape
    out = []
    for b in range(B):
        n, a = int(seq_len[b]), min(max(int(count[b]), 0), T)
        kc = slots_of(k, table[b], n)
        s = np.zeros((Hq // group, n))
        qk = top = 0.0
        for i in range(a):
            t = int(path[b][i]) if path is not None else i
            if not 0 <= t < T:
                continue
            see = min(max(n - a + i + 1, 0), n) if causal else n
            for h in range(Hq):
                if lse[b, h, t] == -np.inf or see == 0:
                    continue
                kk = kc[h // group, :see]
                s[h // group, :see] += np.exp(scale * (kk @ q[b, h, t]) - lse[b, h, t])
                qk = max(qk, scale * (np.abs(kk) @ np.abs(q[b, h, t])).max())
                top = max(top, abs(lse[b, h, t]))
        out.append((s, qk, top))
    return out


def choose(weight, pos, n, keep, first, last, next_pos):
    """(freed slots below keep, kept slots at or above it), in order."""
    if n <= keep:
        return [], []
    def rank(s):
        safe = pos[s] < first or (last > 0 and pos[s] >= next_pos - last)
        w = float(weight[s])
        return (not safe, not np.isnan(w), 0.0 if np.isnan(w) else -w, s)
    kept = set(sorted(range(n), key=rank)[:keep])
    return [s for s in range(keep) if s not in kept], [s for s in range(keep, n) if s in kept]
