"""The cache kernels where a CTA takes many steps of a unit, against float64: running maxima that grow, accumulators
that are rescaled, rings that wrap, sums that are handed over, several units a CTA.

Each test works out from the schedule's rule (equal shares of all steps, one CTA per SM) how many steps a CTA gets,
and asserts it, so that a change of the schedule cannot make it a test of single steps.

Tolerances are those of test_cache_gpu.py, from the arithmetic; the references are plain float64 torch on the GPU.
For the weights the depth of a sum counts: a tile's rows are 16 additions deep in each of 8 parts, which are joined
by 3; then come one addition for each tile of query rows, 3 between the groups, one for each CTA that has a part
(not more than tiles) and the one to the weight:
    |out - ref| <= (2 e + 2^-20 (1 + max |lse|) + (24 + 2 tiles) 2^-24) sum + 2^-23 |ref|
"""
import numpy as np
import pytest
import torch

from test_cache_gpu import U, check_attention, fa, ints, make_tree, normal, np64, pytestmark  # noqa: F401

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def segments(unit_steps):
    """(unit, steps, whether they are the unit's last) of every CTA's share of a line of units."""
    total = sum(unit_steps)
    grid = min(total, torch.cuda.get_device_properties(0).multi_processor_count, 160)
    out = []
    starts = np.concatenate([[0], np.cumsum(unit_steps)])
    for c in range(grid):
        lo, hi = total * c // grid, total * (c + 1) // grid
        for u in range(int(np.searchsorted(starts, lo, "right")) - 1, len(unit_steps)):
            if starts[u] >= hi:
                break
            a, b = max(lo, int(starts[u])), min(hi, int(starts[u + 1]))
            out.append((u, b - a, b == starts[u + 1]))
    return out


def paged(g, per_seq, page, dtype, D):
    """Pools and table for the keys and values [Hkv, n, D] of each sequence; NaN and infinities where nobody is."""
    B, Hkv = len(per_seq), per_seq[0][0].shape[0]
    per = max(1, max(-(-k.shape[1] // page) for k, _ in per_seq))
    num = B * per + 2
    table = torch.randperm(num, generator=g)[:B * per].reshape(B, per)
    pools = []
    for i in range(2):
        x = torch.full((num, Hkv, page, D), float("nan"), dtype=DT[dtype])
        x[..., 1::2] = float("inf")
        for b, kv in enumerate(per_seq):
            n = kv[i].shape[1]
            for c in range(0, n, page):
                m = min(page, n - c)
                x[table[b, c // page], :, :m] = kv[i][:, c:c + m]
        pools.append(x)
    return pools[0], pools[1], table.to(torch.int32)


def attend64(q, kn, vn, per_seq, parent, drafts, scale):
    """o, lse and the bound's ingredients (as cache_oracle.attend), a sequence and KV head at a time."""
    B, Hq, T, D = q.shape
    Hkv = kn.shape[1]
    group = Hq // Hkv
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    pv, av, qk = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    cpu = lambda x: x.reshape(group, t, *x.shape[1:]).cpu().numpy()  # noqa: E731
    for b in range(B):
        t, n = drafts[b], per_seq[b][0].shape[1]
        if t == 0:
            continue
        see = torch.zeros(T, n + t, dtype=torch.bool)
        see[:, :n] = True
        for i in range(t):
            j = i
            while j >= 0:
                see[i, n + j] = True
                j = int(parent[b][j])
        see = see[:t].repeat(group, 1).cuda()
        for c in range(Hkv):
            h = slice(c * group, (c + 1) * group)
            rows = q[b, h, :t].reshape(-1, D).double().cuda()
            k, v = (torch.cat([per_seq[b][i][c], x[b, c, :t]]).double().cuda() for i, x in ((0, kn), (1, vn)))
            s = (rows @ k.T * scale).masked_fill(~see, -float("inf"))
            p = torch.softmax(s, 1)
            o[b, h, :t], lse[b, h, :t] = cpu(p @ v), cpu(torch.logsumexp(s, 1))
            pv[b, h, :t], av[b, h, :t] = cpu(p @ v.abs()), cpu(see.double() @ v.abs())
            qk[b, h, :t] = cpu((rows.abs() @ k.abs().T * scale).masked_fill(~see, 0).amax(1))
    return o, lse, pv, av, qk


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hq,Hkv,T,B", [(64, 8, 4, 4, 16), (128, 8, 4, 4, 16), (256, 8, 4, 4, 16), (64, 4, 2, 70, 32), (128, 4, 2, 70, 32),
                                          (256, 2, 1, 70, 32)])
def test_tree_maxima_that_grow_with_every_step(fa, dtype, D, Hq, Hkv, T, B):  # noqa: F811
    """The scores of each key step lie 9.6 above the last one's (13.8 in log2 units; the accumulator is rescaled beyond
    12), so that every step but a segment's first rescales; the last cached step has one to three keys, so that what was
    rescaled is about a hundredth of the result.  Drafted tokens lie just below the last step, or another 9.6 above it.
    T = 70: more than 128 rows, two row tiles side by side (D <= 128)."""
    g = torch.Generator().manual_seed(100 + D + T)
    BN = 64 if D == 256 else 128
    tiles = [9 + b % 4 for b in range(B)]
    lens = [BN * t + 1 + b % 3 for b, t in enumerate(tiles)]
    drafts = [T - b % 3 for b in range(B)]
    units = (Hq // Hkv * T + 255) // 256 if Hq // Hkv * T > 128 and D != 256 else (Hq // Hkv * T + 127) // 128
    steps = [t + 1 + -(-d // BN) for t, d in zip(tiles, drafts) for _ in range(Hkv * units)]
    cut = segments(steps)
    assert sum(k >= 4 for _, k, _ in cut) >= 100 and sum(k >= 4 and end for _, k, end in cut) >= 20
    root = D ** 0.5
    per_seq = []
    for n in lens:
        k, v = normal(g, (Hkv, n, D), dtype), normal(g, (Hkv, n, D), dtype)
        k[..., 0] = (9.6 * (torch.arange(n) // BN)).to(DT[dtype])
        per_seq.append((k, v))
    q, kn, vn = normal(g, (B, Hq, T, D), dtype, 0.3), normal(g, (B, Hkv, T, D), dtype), normal(g, (B, Hkv, T, D), dtype)
    q[..., 0] = root
    for b, t in enumerate(tiles):
        kn[b, ..., 0] = 9.6 * t + (9.6 if b % 2 else -2.0)
        kn[b, :, drafts[b]:], vn[b, :, drafts[b]:] = float("nan"), float("inf")
    parent = np.stack([make_tree(g, T, "tree") for _ in range(B)])
    kp, vp, table = paged(g, per_seq, 64, dtype, D)
    cache = fa.KVCache(kp.cuda(), vp.cuda(), ints(lens), table.cuda())
    o, lse = torch.full_like(q, 7).cuda(), torch.full((B, Hq, T), 9.0).cuda()
    fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent), draft_len=ints(drafts), o=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)
    ref = attend64(q, kn, vn, per_seq, parent, drafts, 1 / root)
    check_attention(o, lse, ref, dtype, drafts, f"{dtype} D{D} T{T}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hq,Hkv,T,B,n", [(64, 16, 2, 5, 6, 9000), (128, 16, 2, 5, 6, 9000), (256, 16, 2, 5, 3, 9000), (64, 8, 2, 40, 6, 9000),
                                            (128, 8, 2, 40, 6, 9000), (128, 32, 4, 64, 2, 9000)])
def test_tree_long_runs_of_random_scores(fa, dtype, D, Hq, Hkv, T, B, n):  # noqa: F811
    """Five steps a CTA and more, units that are cut, scores of tens (the maximum grows at random)."""
    g = torch.Generator().manual_seed(200 + D + T)
    BN, rows = 64 if D == 256 else 128, Hq // Hkv * T
    lens = [n - 701 * b for b in range(B)]
    units = -(-rows // (256 if rows > 128 and D != 256 else 128))
    cut = segments([-(-x // BN) + -(-T // BN) for x in lens for _ in range(Hkv * units)])
    assert sum(k >= 4 for _, k, _ in cut) >= 100
    per_seq = [(normal(g, (Hkv, x, D), dtype, 2.5), normal(g, (Hkv, x, D), dtype)) for x in lens]
    q, kn, vn = normal(g, (B, Hq, T, D), dtype, 2.5), normal(g, (B, Hkv, T, D), dtype, 2.5), normal(g, (B, Hkv, T, D), dtype)
    parent = np.stack([make_tree(g, T, "tree") for _ in range(B)])
    kp, vp, table = paged(g, per_seq, 48, dtype, D)
    cache = fa.KVCache(kp.cuda(), vp.cuda(), ints(lens), table.cuda())
    o, lse = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent))
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)
    check_attention(o, lse, attend64(q, kn, vn, per_seq, parent, [T] * B, D ** -0.5), dtype, [T] * B, f"{dtype} D{D} T{T}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_tokens_with_two_row_tiles(fa, dtype, D):  # noqa: F811
    """More than 128 rows a KV head: a drafted token with NaN or infinities reaches the rows that see it, as what it is,
    and no others, in both row tiles."""
    g = torch.Generator().manual_seed(5)
    B, Hq, Hkv, T = 1, 80, 2, 6                                       # 240 rows
    per_seq = [(normal(g, (Hkv, 150, D), dtype), normal(g, (Hkv, 150, D), dtype))]
    k, v, table = paged(g, per_seq, 16, dtype, D)
    q, kn, vn = (normal(g, (B, h, T, D), dtype) for h in (Hq, Hkv, Hkv))
    parent = np.array([[-1, 0, 0, 1, 2, 2]])
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([150]), table.cuda())
    o2, lse2 = (np64(x) for x in fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent)))
    check_attention(torch.tensor(o2), torch.tensor(lse2), attend64(q, kn, vn, per_seq, parent, [T], D ** -0.5), dtype, [T], "clean")
    vn[0, :, 1, 3], vn[0, :, 1, 9] = float("inf"), float("nan")      # seen by 1 and 3
    vn[0, :, 4, D - 1] = float("-inf")                               # seen by 4
    kn[0, :, 5] = float("nan")                                       # seen by 5
    o, lse = (np64(x) for x in fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent)))
    assert fa.fa_device_status() == (0, 0)
    for t in (0, 2):
        assert (o[:, :, t] == o2[:, :, t]).all() and (lse[:, :, t] == lse2[:, :, t]).all()
    for t in (1, 3):
        assert (o[:, :, t, 3] == np.inf).all() and np.isnan(o[:, :, t, 9]).all()
        rest = [d for d in range(D) if d not in (3, 9)]
        assert (o[:, :, t][..., rest] == o2[:, :, t][..., rest]).all()
    assert (o[:, :, 4, D - 1] == -np.inf).all() and (o[:, :, 4, :D - 1] == o2[:, :, 4, :D - 1]).all()
    assert np.isnan(o[:, :, 5]).all() and np.isnan(lse[:, :, 5]).all()


def test_sequences_share_pages_that_are_read(fa):  # noqa: F811
    """Two sequences with the pages of a common prefix, one of them twice in a table: each attends over its own slots."""
    g = torch.Generator().manual_seed(6)
    Hq, Hkv, D, T, page = 4, 2, 128, 3, 16
    k, v = normal(g, (9, Hkv, page, D), "bf16"), normal(g, (9, Hkv, page, D), "bf16")
    table = np.array([[3, 5, 0, 7], [3, 5, 5, 2]])
    lens = [55, 61]
    per_seq = [tuple(x[torch.tensor(row)].transpose(0, 1).reshape(Hkv, -1, D)[:, :n] for x in (k, v)) for row, n in zip(table, lens)]
    q, kn, vn = (normal(g, (2, h, T, D), "bf16") for h in (Hq, Hkv, Hkv))
    o, lse = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), fa.KVCache(k.cuda(), v.cuda(), ints(lens), ints(table)))
    parent = np.tile(np.arange(T) - 1, (2, 1))
    check_attention(o, lse, attend64(q, kn, vn, per_seq, parent, [T, T], D ** -0.5), "bf16", [T, T], "shared pages")


# ---------------------------------------------------------------- accumulated weights

def weigh64(q, lse, k, n, rows, count, scale, group, causal):
    """sum over the heads of each KV head and the counted rows of exp(scale q.k - lse): [Hkv, n] float64, of one sequence;
    the largest scale sum |q||k| and |lse|."""
    Hkv = k.shape[0]
    out, qk, top = torch.zeros(Hkv, n, dtype=torch.float64, device="cuda"), 0.0, 0.0
    see = torch.arange(n, device="cuda")[None] < (n - count + 1 + torch.arange(count, device="cuda"))[:, None] if causal else None
    for h in range(q.shape[0]):
        c = h // group
        x, l = q[h, rows].double().cuda(), lse[h, rows].double().cuda()
        p = torch.exp(x @ k[c].double().cuda().T * scale - l[:, None])
        out[c] += (p.masked_fill(~see, 0) if causal else p).sum(0)
        qk = max(qk, float((x.abs() @ k[c].double().cuda().abs().T).max()) * scale)
        top = max(top, float(l.abs().max()))
    return out.cpu().numpy(), qk, top


def run(fa, dtype, Hq, Hkv, D, lens, counts, T, page, with_path=False, causal=True, least=10, seed=1):  # noqa: F811
    g = torch.Generator().manual_seed(seed)
    B, group = len(lens), Hq // Hkv
    NQ = 64 if D == 256 else 128
    heads = T >= 128 and not with_path
    keys = 256 if heads else 128
    steps = []
    for n, a in zip(lens, counts):
        for kt in range(-(-n // keys)):
            if heads:
                first = max(0, (kt * keys - (n - a)) // NQ) if causal else 0
                one = group * (-(-a // NQ) - first)
            else:
                one = -(-group * (a if with_path else T) // NQ)
            steps.append(one)
    steps = [x for b in range(B) for _ in range(Hkv)
             for x in steps[sum(-(-m // keys) for m in lens[:b]):sum(-(-m // keys) for m in lens[:b + 1])]]
    assert sum(steps) >= least * torch.cuda.get_device_properties(0).multi_processor_count
    if not heads:   # key tiles of several query tiles, completed by one CTA: sums are handed over again and again
        whole = [k for u, k, end in segments(steps) if k == steps[u]]
        assert min(steps) >= 2 and len(whole) >= 100
    per_seq = [(normal(g, (Hkv, n, D), dtype), normal(g, (Hkv, n, D), dtype)) for n in lens]
    k, v, table = paged(g, per_seq, page, dtype, D)
    q = normal(g, (B, Hq, T, D), dtype)
    lse = torch.randn(B, Hq, T, generator=g) + 4.0
    rows = [torch.randperm(T, generator=g)[:a] if with_path else torch.arange(a) for a in counts]
    path = None
    if with_path:
        path = np.full((B, T), -1)
        for b, r in enumerate(rows):
            path[b, :len(r)] = r.numpy()
    for b, r in enumerate(rows):                     # rows that do not count hold anything
        off = torch.ones(T, dtype=torch.bool)
        off[r] = False
        q[b, :, off], lse[b, :, off] = float("nan"), float("nan")
    cap = table.shape[1] * page
    weight = torch.rand(B, Hkv, cap, generator=g)
    out = torch.full((B, Hkv, cap), -3.0).cuda()
    fa.cache_weights(fa.KVCache(k.cuda(), v.cuda(), ints(lens), table.cuda()), q.cuda(), lse.cuda(), weight.cuda(),
                     path=None if path is None else ints(path), count=ints(counts), causal=causal, out=out)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)
    got, w = np64(out), np64(weight)
    for b, n in enumerate(lens):
        total, qk, top = weigh64(q[b], lse[b], per_seq[b][0], n, rows[b], counts[b], D ** -0.5, group, causal)
        want = total + w[b, :, :n]
        tiles = -(-group * counts[b] // NQ) + group
        tol = (2.0 ** -17 * qk + 2.0 ** -20 * (1 + top) + (24 + 2 * tiles) * 2.0 ** -24) * total + 2.0 ** -23 * np.abs(want)
        far = np.abs(got[b, :, :n] - want) - tol
        assert np.isfinite(got[b, :, :n]).all() and far.max() <= 1e-12, f"sequence {b}: {far.max():.3e} outside"
        assert (got[b, :, n:] == -3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("with_path", [False, True])
@pytest.mark.parametrize("group,T,B", [(2, 127, 60), (4, 90, 40), (8, 120, 24)])
def test_weights_hand_their_sums_over(fa, dtype, D, with_path, group, T, B):  # noqa: F811
    """Key tiles of 2 to 15 query tiles, several of them a CTA: the four groups' sums are joined for each."""
    lens = [1100 + 31 * (b % 7) for b in range(B)]
    counts = [T - (b % 3 if with_path else b % 5) for b in range(B)]
    run(fa, dtype, 2 * group, 2, D, lens, counts, T, 48, with_path=with_path, causal=group != 4, seed=D + T)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_weights_of_prompts_with_many_steps(fa, dtype, D, causal):  # noqa: F811
    """Ten and more steps a CTA in the prompt kernel: K pairs replaced in tensor memory, rings that wrap."""
    run(fa, dtype, 8, 2, D, [1500, 1100, 2000, 1301, 1777, 1408], [1500, 1000, 1990, 1301, 1500, 1280], 2000, 16, causal=causal, seed=D)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_of_long_prompts(fa, dtype, D):  # noqa: F811
    """The variant for 4096 tokens and more, with grouped heads."""
    run(fa, dtype, 4, 2, D, [4200, 4500], [4200, 4096], 4300, 80, seed=D)
