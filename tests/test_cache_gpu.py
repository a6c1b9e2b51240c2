"""GPU tests of the cache operators against the float64 oracle (cache_oracle.py).

Tolerances, from the arithmetic.  u = eps / 2 is the type's rounding (2^-8 bf16, 2^-11 fp16).

  attention   A score is an fp32 sum of exact products: its error is at most 2^-18 sum |q||k| scale =: e
              (2^-24 for each of up to 256 additions in the worst order, and the scale's own rounding).
              exp turns it into a relative error e of each weight, and the same again in the sum; the
              hardware exponential adds 2^-21.  Each weight is rounded to the type for P V (u), the
              result once more (u):
                  |o - ref| <= u |ref| + (u + 2 e + 2^-20) sum_j p_j |v_j|
              fp16 weights below 2^-14 are rounded to multiples of 2^-24 of the largest weight: with at
              least one weight of 1, half a step is 2^-25 sum_j |v_j| more.
                  |lse - ref| <= e + 2^-20 (1 + |ref|)
  append      a copy: equal.
  weights     every term has the score's error e, the rounding of lse and of the exponent (2^-22 (1 + |lse|))
              and the exponential's (2^-21); a sum of up to 32 tiles of 128 rows is at most 64 additions
              deep (2^-18), the addition to the weight one more:
                  |out - ref| <= (2 e + 2^-20 (1 + max |lse|) + 2^-18) sum + 2^-23 |ref|
  eviction    copies and whole numbers: equal.
"""
import numpy as np
import pytest
import torch

from cache_oracle import attend, choose, weigh
from programming_flashattention_fwd_gb300 import build as fa_build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fa_build.build()
    import programming_flashattention_fwd_gb300 as pkg
    return pkg


def np64(t):
    return t.detach().double().cpu().numpy()


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make_pool(g, lens, Hkv, D, page, dtype, room=0, dense=False, std=1.0):
    """A pool whose pages are shared out at random; every slot that no sequence uses holds NaN or infinity."""
    B = len(lens)
    per = max(1, -(-(max(lens) + room) // page))
    num = B * per + (0 if dense else 2)
    table = torch.arange(B * per).reshape(B, per) if dense else torch.randperm(num, generator=g)[:B * per].reshape(B, per)
    k = torch.full((num, Hkv, page, D), float("nan"), dtype=DT[dtype])
    v = torch.full_like(k, float("nan"))
    v[..., ::2] = float("inf")
    for b, n in enumerate(lens):
        for c in range(0, n, page):
            m = min(page, n - c)
            k[table[b, c // page], :, :m] = normal(g, (Hkv, m, D), dtype, std)
            v[table[b, c // page], :, :m] = normal(g, (Hkv, m, D), dtype)
    return k, v, table.to(torch.int32)


def make_tree(g, T, kind):
    if kind == "chain":
        return np.arange(T) - 1
    if kind == "star":
        return np.full(T, -1)
    parent = np.full(T, -1)
    for t in range(1, T):
        r = torch.randint(0, 100, (2,), generator=g).tolist()
        parent[t] = -1 if r[0] < 8 else t - 1 - min(t - 1, r[1] % 5)
    return parent


def check_attention(o, lse, ref, dtype, draft_len, what):
    ro, rl, pv, av, qk = ref
    o, lse = np64(o), np64(lse)
    e = 2.0 ** -18 * qk
    tol = U[dtype] * np.abs(ro) + (U[dtype] + 2 * e[..., None] + 2.0 ** -20) * pv + (2.0 ** -25 * av if dtype == "fp16" else 0)
    for b, t in enumerate(draft_len):
        assert np.isfinite(o[b, :, :t]).all() and np.isfinite(lse[b, :, :t]).all(), what
        far = np.abs(o[b, :, :t] - ro[b, :, :t]) - tol[b, :, :t]
        assert far.size == 0 or far.max() <= 1e-12, f"{what}: sequence {b}: o is {far.max():.3e} outside"
        far = np.abs(lse[b, :, :t] - rl[b, :, :t]) - e[b, :, :t] - 2.0 ** -20 * (1 + np.abs(rl[b, :, :t]))
        assert far.size == 0 or far.max() <= 0, f"{what}: sequence {b}: lse is {far.max():.3e} outside"
        # rows behind draft_len are left as they were
        assert (o[b, :, t:] == 7).all() and (lse[b, :, t:] == 9).all(), what


def run_tree(fa, dtype, Hq, Hkv, D, lens, drafts, T, page, kind="tree", dense=False, std=1.0, seed=1, use_len=True):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    k, v, table = make_pool(g, lens, Hkv, D, page, dtype, dense=dense, std=std)
    q = normal(g, (B, Hq, T, D), dtype, std)
    kn, vn = normal(g, (B, Hkv, T, D), dtype, std), normal(g, (B, Hkv, T, D), dtype)
    for b, t in enumerate(drafts):   # padding behind draft_len is never read as a key
        kn[b, :, t:], vn[b, :, t:] = float("nan"), float("inf")
    parent = np.stack([make_tree(g, T, kind) for _ in range(B)])
    cache = fa.KVCache(k.cuda(), v.cuda(), ints(lens), None if dense else table.cuda())
    o, lse = torch.full_like(q, 7).cuda(), torch.full((B, Hq, T), 9.0).cuda()
    fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=None if kind == "chain" else ints(parent),
                      draft_len=ints(drafts) if use_len else None, o=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)
    ref = attend(np64(q), np64(kn), np64(vn), np64(k), np64(v), table.numpy(), lens, parent, drafts, 1 / np.sqrt(D))
    check_attention(o, lse, ref, dtype, drafts, f"{dtype} Hq{Hq} Hkv{Hkv} D{D} {lens} {drafts} T{T} page{page} {kind}")


HEADS = [(4, 1), (3, 3), (8, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS)
def test_tree_ragged(fa, dtype, D, heads):
    """Empty, one-slot, page-end and tile-end caches side by side; drafts of zero, one and all tokens."""
    run_tree(fa, dtype, *heads, D, [0, 1, 16, 127, 128, 129, 200, 37], [7, 7, 0, 1, 3, 7, 5, 2], 7, 16)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256, 272])
def test_tree_pages(fa, page):
    run_tree(fa, "bf16", 4, 2, 128, [page - 1, 300, 2 * page, page + 1], [5, 4, 5, 1], 5, page, seed=page)


MANY_PAGES = [(64, 16), (128, 16), (128, 48), (256, 16), (64, 80)]


@pytest.mark.parametrize("D,page", MANY_PAGES)
def test_tree_many_small_pages(fa, D, page):
    """A CTA's run of keys takes more pages than are looked up at a time, from any place in a group of them."""
    lens = [1000 + 53 * i for i in range(20)]
    run_tree(fa, "bf16", 8, 8, D, lens, [1 + i % 2 for i in range(20)], 2, page, seed=D + page)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_dense_cache(fa, D):
    run_tree(fa, "fp16", 4, 2, D, [100, 161, 0], [3, 2, 3], 3, 176, dense=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,kind", [(1, "tree"), (1, "chain"), (2, "star"), (33, "chain"), (64, "tree"), (130, "tree"), (130, "chain")])
def test_tree_shapes(fa, D, T, kind):
    """One token; several row tiles; drafted tokens over more than one key tile."""
    run_tree(fa, "bf16", 8, 2, D, [90, 257], [T, max(1, T - 1)], T, 32, kind=kind, seed=T)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_long_cache_is_cut(fa, D):
    """One sequence whose keys are shared out over many CTAs, beside short ones."""
    run_tree(fa, "bf16", 2, 1, D, [6001, 3, 500], [2, 3, 1], 3, 64)


def test_tree_many_sequences(fa):
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 150, 70)]
    run_tree(fa, "bf16", 2, 2, 64, lens, [1 + i % 3 for i in range(70)], 3, 16)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_large_logits(fa, dtype, D):
    """Scores of tens: the running maximum grows past the rescaling threshold again and again."""
    run_tree(fa, dtype, 4, 1, D, [900, 40], [6, 5], 6, 16, std=3.0)


def test_tree_without_draft_len(fa):
    run_tree(fa, "bf16", 4, 2, 128, [50, 70], [4, 4], 4, 16, use_len=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_non_finite_tokens_stay_on_their_branch(fa, dtype, D):
    """A drafted token with NaN or infinities in its key or value reaches the rows that see it, as what
    it is, and no others."""
    g = torch.Generator().manual_seed(5)
    B, Hq, Hkv, T = 1, 4, 2, 6
    k, v, table = make_pool(g, [150], Hkv, D, 16, dtype)
    q, kn, vn = (normal(g, (B, h, T, D), dtype) for h in (Hq, Hkv, Hkv))
    parent = np.array([[-1, 0, 0, 1, 2, 2]])
    clean = (kn.clone(), vn.clone())
    vn[0, :, 1, 3], vn[0, :, 1, 9] = float("inf"), float("nan")      # seen by 1 and 3
    vn[0, :, 4, D - 1] = float("-inf")                               # seen by 4
    kn[0, :, 5] = float("nan")                                       # seen by 5
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([150]), table.cuda())
    o, lse = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent))
    o2, lse2 = fa.tree_attention(q.cuda(), clean[0].cuda(), clean[1].cuda(), cache, parent=ints(parent))
    torch.cuda.synchronize()
    o, o2, lse, lse2 = np64(o), np64(o2), np64(lse), np64(lse2)
    for t in (0, 2):
        assert (o[:, :, t] == o2[:, :, t]).all() and (lse[:, :, t] == lse2[:, :, t]).all()
    for t in (1, 3):
        assert (o[:, :, t, 3] == np.inf).all() and np.isnan(o[:, :, t, 9]).all()
        rest = [d for d in range(D) if d not in (3, 9)]
        assert (o[:, :, t][..., rest] == o2[:, :, t][..., rest]).all()
    assert (o[:, :, 4, D - 1] == -np.inf).all() and (o[:, :, 4, :D - 1] == o2[:, :, 4, :D - 1]).all()
    assert np.isnan(o[:, :, 5]).all() and np.isnan(lse[:, :, 5]).all()


def test_tree_broken_parents_are_roots(fa):
    """An entry that does not come before its child ends the path: here every token sees itself alone."""
    g = torch.Generator().manual_seed(6)
    k, v, table = make_pool(g, [20], 1, 64, 16, "bf16")
    q, kn, vn = (normal(g, (1, 1, 4, 64), "bf16").cuda() for _ in range(3))
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([20]), table.cuda())
    a = fa.tree_attention(q, kn, vn, cache, parent=ints([[0, 5, 2, 1 << 30]]))
    b = fa.tree_attention(q, kn, vn, cache, parent=ints([[-1, -1, -1, -1]]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_matches_the_forward_over_a_dense_cache(fa):
    """A chain over a cache is the bottom-right causal forward over all keys."""
    g = torch.Generator().manual_seed(7)
    B, Hq, Hkv, D, n, T = 2, 8, 2, 128, 320, 24
    k, v = normal(g, (B, Hkv, n + T, D), "bf16").cuda(), normal(g, (B, Hkv, n + T, D), "bf16").cuda()
    q = normal(g, (B, Hq, T, D), "bf16").cuda()
    o1, l1 = fa.attention(q, k, v, causal=2)
    cache = fa.KVCache(k[:, :, :n].contiguous(), v[:, :, :n].contiguous(), ints([n, n]))
    o2, l2 = fa.tree_attention(q, k[:, :, n:].contiguous(), v[:, :, n:].contiguous(), cache)
    assert (o1.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * (1 + o1.float().abs().max())
    assert (l1 - l2).abs().max() <= 2e-5


def test_append(fa):
    g = torch.Generator().manual_seed(8)
    B, Hkv, D, T, page, cap = 3, 2, 128, 6, 16, 48
    lens, count = [0, 15, 45], [4, 6, 6]
    k, v, table = make_pool(g, [cap] * B, Hkv, D, page, "bf16")
    kn, vn = normal(g, (B, Hkv, T, D), "bf16"), normal(g, (B, Hkv, T, D), "bf16")
    path = np.array([[1, 2, 4, 5, -1, -1], [0, 1, 2, 3, 4, 5], [5, 5, 0, 1, 2, 3]])
    start = [100, 7, 1]
    kd, vd = k.cuda(), v.cuda()
    weight, pos = torch.full((B, Hkv, cap), 3.0).cuda(), torch.full((B, Hkv, cap), -5, dtype=torch.int32).cuda()
    fa.cache_append(fa.KVCache(kd, vd, ints(lens), table.cuda()), kn.cuda(), vn.cuda(), path=ints(path), count=ints(count), weight=weight,
                    pos=pos, start=ints(start))
    w, ps = torch.full((B, Hkv, cap), 3.0), torch.full((B, Hkv, cap), -5, dtype=torch.int32)
    for b in range(B):
        for i in range(count[b]):
            s = lens[b] + i
            if s >= cap:
                continue    # behind the capacity: dropped
            k[table[b, s // page], :, s % page] = kn[b, :, path[b, i]]
            v[table[b, s // page], :, s % page] = vn[b, :, path[b, i]]
            w[b, :, s], ps[b, :, s] = 0, start[b] + i
    assert torch.equal(kd.cpu().view(torch.int16), k.view(torch.int16)) and torch.equal(vd.cpu().view(torch.int16), v.view(torch.int16))
    assert torch.equal(weight.cpu(), w) and torch.equal(pos.cpu(), ps)


@pytest.mark.parametrize("D", [64, 256])
def test_append_everything_in_order(fa, D):
    g = torch.Generator().manual_seed(9)
    B, Hkv, T, page = 2, 3, 77, 32
    k, v, table = make_pool(g, [0] * B, Hkv, D, page, "fp16", room=T)
    kn, vn = normal(g, (B, Hkv, T, D), "fp16"), normal(g, (B, Hkv, T, D), "fp16")
    kd, vd = k.cuda(), v.cuda()
    fa.cache_append(fa.KVCache(kd, vd, ints([0, 0]), table.cuda()), kn.cuda(), vn.cuda())
    for b in range(B):
        for s in range(T):
            k[table[b, s // page], :, s % page], v[table[b, s // page], :, s % page] = kn[b, :, s], vn[b, :, s]
    assert torch.equal(kd.cpu().view(torch.int16), k.view(torch.int16)) and torch.equal(vd.cpu().view(torch.int16), v.view(torch.int16))


def test_a_page_that_does_not_exist(fa):
    """Table entries outside the pool: their slots read as zeros, writes to them are dropped."""
    g = torch.Generator().manual_seed(10)
    k, v, table = make_pool(g, [48], 1, 64, 16, "bf16")
    q, kn, vn = (normal(g, (1, 1, 2, 64), "bf16") for _ in range(3))
    for bad in (-1, k.shape[0], 1 << 30):
        t2 = table.clone()
        t2[0, 1] = bad
        kd, vd = k.cuda(), v.cuda()
        cache = fa.KVCache(kd, vd, ints([48]), t2.cuda())
        o, lse = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache)
        zk, zv = k.clone(), v.clone()
        zk[table[0, 1]], zv[table[0, 1]] = 0, 0
        ref = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), fa.KVCache(zk.cuda(), zv.cuda(), ints([48]), table.cuda()))
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
        fa.cache_append(fa.KVCache(kd, vd, ints([17]), t2.cuda()), kn.cuda(), vn.cuda())
        torch.cuda.synchronize()
        assert torch.equal(kd.cpu().view(torch.int16), k.view(torch.int16))


# ---------------------------------------------------------------- accumulated weights

def run_weights(fa, dtype, Hq, Hkv, D, lens, counts, T, page, path=None, causal=True, seed=1, kind="out", poison=True, std=1.0):
    g = torch.Generator().manual_seed(seed)
    B, group = len(lens), Hq // Hkv
    k, v, table = make_pool(g, lens, Hkv, D, page, dtype)
    cap = table.shape[1] * page
    q = normal(g, (B, Hq, T, D), dtype, std)
    lse = torch.randn(B, Hq, T, generator=g) + 4.0
    if path is not None:
        path = np.asarray(path)
    if T > 3:
        lse[:, 0, 2] = -float("inf")      # a row that saw nothing
    if poison:                            # rows that do not count hold anything
        for b, a in enumerate(counts):
            used = set(range(min(max(a, 0), T)) if path is None else [int(x) for x in path[b][:max(a, 0)]])
            for t in range(T):
                if t not in used:
                    q[b, :, t], lse[b, :, t] = float("nan"), float("nan")
    w = torch.rand(B, Hkv, cap, generator=g)
    cache = fa.KVCache(k.cuda(), v.cuda(), ints(lens), table.cuda())
    weight = None if kind == "none" else w.cuda()
    out = torch.full((B, Hkv, cap), -3.0).cuda() if kind != "in place" else None
    got = fa.cache_weights(cache, q.cuda(), lse.cuda(), weight, path=None if path is None else ints(path), count=ints(counts),
                           causal=causal, out=out)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)
    assert got is (weight if kind == "in place" else out)
    what = f"{dtype} Hq{Hq} Hkv{Hkv} D{D} {lens} {counts} T{T} page{page} {kind}"
    ref = weigh(np64(q), np64(lse), np64(k), table.numpy(), lens, path, counts, causal, 1 / np.sqrt(D), group)
    got, w = np64(got), np64(w)
    for b, n in enumerate(lens):
        total, qk, top = ref[b]
        want = total + (0 if kind == "none" else w[b, :, :n])
        tol = (2.0 ** -17 * qk + 2.0 ** -20 * (1 + top) + 2.0 ** -18) * total + 2.0 ** -23 * np.abs(want)
        far = np.abs(got[b, :, :n] - want) - tol
        assert np.isfinite(got[b, :, :n]).all() and (far.size == 0 or far.max() <= 1e-12), f"{what}: sequence {b}: {far.max():.3e} outside"
        # slots that are not in use are left as they were
        assert (got[b, :, n:] == (w[b, :, n:] if kind == "in place" else -3.0)).all(), what


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS)
def test_weights_of_prompts(fa, dtype, D, heads):
    """Long enough for the tiles of one head; counts of zero, one and more than there are slots."""
    run_weights(fa, dtype, *heads, D, [0, 1, 130, 300, 128, 70], [0, 1, 130, 200, 5, 90], 210, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 7, 50, 127, 128, 129])
@pytest.mark.parametrize("causal", [True, False])
def test_weights_of_short_prompts(fa, D, T, causal):
    run_weights(fa, "bf16", 8, 2, D, [400, 129, T], [T, max(1, T - 3), T], T, 48, causal=causal, seed=T)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["out", "in place", "none"])
def test_weights_of_accepted_tokens(fa, dtype, D, kind):
    path = [[0, 2, 5, 8, -1, -1, -1, -1, -1], [8, -1, -1, -1, -1, -1, -1, -1, -1], list(range(9)), [-1] * 9, [3, 99, -7, 4, -1, -1, -1, -1, -1]]
    run_weights(fa, dtype, 8, 2, D, [260, 500, 128, 40, 77], [4, 1, 9, 0, 4], 9, 32, path=path, kind=kind)


def test_weights_of_many_accepted_tokens(fa):
    """More gathered rows than one tile holds, and a row that counts twice."""
    T = 70
    run_weights(fa, "bf16", 8, 2, 128, [300, 200], [70, 40], T, 16, path=[list(range(T)), [0, 0] + list(range(1, T - 1))])


@pytest.mark.parametrize("D,page", MANY_PAGES)
@pytest.mark.parametrize("with_path", [False, True])
def test_weights_many_small_pages(fa, D, page, with_path):
    lens = [1000 + 53 * i for i in range(20)]
    run_weights(fa, "bf16", 8, 8, D, lens, [2] * 20, 2, page, path=[[1, 0]] * 20 if with_path else None, seed=D + page)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_cut_among_ctas(fa, D):
    """Fewer key tiles than CTAs, many query tiles: key tiles are computed in parts."""
    run_weights(fa, "fp16", 4, 1, D, [900], [900], 900, 128)


def test_weights_with_large_scores(fa):
    run_weights(fa, "bf16", 4, 2, 128, [200, 150], [150, 150], 150, 16, std=3.0)


def test_weights_repeat_exactly(fa):
    g = torch.Generator().manual_seed(3)
    k, v, table = make_pool(g, [700], 2, 128, 16, "bf16")
    q, lse = normal(g, (1, 8, 700, 128), "bf16").cuda(), torch.randn(1, 8, 700, generator=g).cuda() + 5
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([700]), table.cuda())
    first = fa.cache_weights(cache, q, lse)
    for _ in range(5):
        assert torch.equal(fa.cache_weights(cache, q, lse), first)


# ---------------------------------------------------------------- eviction

def run_evict(fa, Hkv, D, lens, keep, page, first=0, last=0, cap=None, weight=None, in_place=True, seed=1, dtype="bf16", dense=False):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    room = 0 if cap is None else cap - max(lens)
    k, v, table = make_pool(g, lens, Hkv, D, page, dtype, room=room, dense=dense)
    cap = table.shape[1] * page
    w = torch.randn(B, Hkv, cap, generator=g) if weight is None else weight(g, (B, Hkv, cap))
    pos = torch.stack([torch.stack([torch.randperm(cap, generator=g) for _ in range(Hkv)]) for _ in range(B)]).to(torch.int32)
    nxt = [n + 3 for n in lens]
    kd, vd, wd, pd = k.cuda(), v.cuda(), w.cuda(), pos.cuda()
    wo, po = (wd, pd) if in_place else (torch.full_like(wd, 5.0), torch.full_like(pd, -9))
    cache = fa.KVCache(kd, vd, ints(lens), None if dense else table.cuda())
    left = fa.cache_evict(cache, wd, pd, keep, first=first, last=last, next_pos=ints(nxt) if last else None,
                          weight_out=None if in_place else wo, pos_out=None if in_place else po)
    torch.cuda.synchronize()
    assert left.tolist() == [min(n, keep) for n in lens]
    rw, rp = (w.clone(), pos.clone()) if in_place else (torch.full_like(w, 5.0), torch.full_like(pos, -9))
    for b, n in enumerate(lens):
        m = min(n, keep)
        for h in range(Hkv):
            dst, src = choose(w[b, h].numpy(), pos[b, h].numpy(), n, keep, first, last, nxt[b])
            assert len(dst) == len(src)
            rw[b, h, :m], rp[b, h, :m] = w[b, h, :m], pos[b, h, :m]
            for d, s in zip(dst, src):
                rw[b, h, d], rp[b, h, d] = w[b, h, s], pos[b, h, s]
                for x in (k, v):
                    x[table[b, d // page], h, d % page] = x[table[b, s // page], h, s % page]
    bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(kd), bits(k)) and torch.equal(bits(vd), bits(v))
    assert torch.equal(wo.cpu().view(torch.int32), rw.view(torch.int32)) and torch.equal(po.cpu(), rp)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (100, 4, 32), (333, 0, 7), (599, 3, 0)])
def test_evict(fa, D, keep, first, last, in_place):
    run_evict(fa, 2, D, [600, 0, 1, keep, keep + 1, 555], keep, 16, first, last, in_place=in_place, seed=keep, dtype="fp16")


@pytest.mark.parametrize("page", [16, 48, 128])
def test_evict_long(fa, page):
    """Clusters of several CTAs."""
    run_evict(fa, 1, 64, [9000, 5000], 3001, page, 4, 64)


def test_evict_dense_cache(fa):
    run_evict(fa, 3, 128, [176, 100], 60, 176, 2, 2, dense=True)


TIES = {
    "all equal": lambda g, s: torch.zeros(s),
    "few values": lambda g, s: torch.randint(-2, 3, s, generator=g).float(),
    "signed zeros": lambda g, s: torch.where(torch.rand(s, generator=g) < 0.5, -0.0, 0.0),
    "infinities and NaN": lambda g, s: torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, 1e-45, -3.4e38])[torch.randint(0, 6, s, generator=g)],
    "one outlier": lambda g, s: torch.where(torch.arange(s[-1]) == 77, 1e30, 1e-30 * torch.rand(s, generator=g)),
}


@pytest.mark.parametrize("kind", list(TIES))
@pytest.mark.parametrize("n", [500, 4000])
def test_evict_ties(fa, kind, n):
    run_evict(fa, 2, 64, [n, n - 77], n // 3, 16, 4, 8, weight=TIES[kind])


def test_evict_nothing(fa):
    run_evict(fa, 2, 64, [50, 3], 64, 16, 4, 8, in_place=False)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("D,page", [(64, 16), (128, 48)])
def test_a_decoding_loop(fa, D, page):
    """Prompt, eviction, then drafting steps: attend, accept, append, weigh, evict.  The oracle keeps every
    head's keys, values, weights and positions in float64 and is told only which tokens were accepted;
    what the cache holds is compared with it at the end of every step."""
    g = torch.Generator().manual_seed(11)
    B, Hq, Hkv, T, keep, first, last = 2, 4, 2, 9, 60, 2, 8
    group, scale = Hq // Hkv, 1 / np.sqrt(D)
    prompt = [90, 75]
    per = -(-130 // page)
    pool = torch.zeros(B * per + 1, Hkv, page, D, dtype=torch.bfloat16).cuda()
    table = torch.randperm(B * per + 1, generator=g)[:B * per].reshape(B, per)
    seq = ints([0, 0])
    cache = fa.KVCache(pool, pool.clone(), seq, ints(table))
    cap = cache.capacity
    weight, pos = torch.zeros(B, Hkv, cap).cuda(), torch.zeros(B, Hkv, cap, dtype=torch.int32).cuda()
    nxt = ints([0, 0])
    P = max(prompt)
    q, kn, vn = (normal(g, (B, h, P, D), "bf16") for h in (Hq, Hkv, Hkv))
    # the prompt: attention of a chain over the empty cache, then its keys and weights
    o, lse = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, draft_len=ints(prompt))
    fa.cache_append(cache, kn.cuda(), vn.cuda(), count=ints(prompt), weight=weight, pos=pos, start=nxt)
    seq += ints(prompt)
    nxt += ints(prompt)
    fa.cache_weights(cache, q.cuda(), lse, weight, count=ints(prompt))
    none = np.zeros((1, Hkv, page, D))
    chain = np.tile(np.arange(P) - 1, (B, 1))
    ref = attend(np64(q), np64(kn), np64(vn), none, none, np.zeros((B, 1), int), [0, 0], chain, prompt, scale)
    state = []     # [b][head]: keys, values, weights, positions in the order of the slots
    for b in range(B):
        state.append([])
        for c in range(Hkv):
            s = dict(k=np64(kn)[b, c, :prompt[b]], v=np64(vn)[b, c, :prompt[b]], w=np.zeros(prompt[b]), p=np.arange(prompt[b]))
            for h in range(c * group, (c + 1) * group):
                for i in range(prompt[b]):
                    s["w"][:i + 1] += np.exp(scale * (s["k"][:i + 1] @ np64(q)[b, h, i]) - ref[1][b, h, i])
            state[b].append(s)

    def evict():
        seq.copy_(fa.cache_evict(cache, weight, pos, keep, first=first, last=last, next_pos=nxt))
        for b in range(B):
            for c in range(Hkv):
                s, n = state[b][c], len(state[b][c]["p"])
                # the choice is the kernel's own: by its weights, which a rounding apart may order otherwise
                kept = set(pos[b, c, :int(seq[b])].tolist())
                assert len(kept) == min(n, keep)
                safe = {int(x) for x in s["p"] if x < first or x >= int(nxt[b]) - last}
                assert safe <= kept
                if n > keep:
                    low = min(s["w"][i] for i in range(n) if int(s["p"][i]) in kept - safe)
                    high = max(s["w"][i] for i in range(n) if int(s["p"][i]) not in kept)
                    assert low >= high * (1 - 1e-3)
                dst = [i for i in range(min(n, keep)) if int(s["p"][i]) not in kept]
                src = [i for i in range(keep, n) if int(s["p"][i]) in kept]
                for x in s:
                    s[x][dst] = s[x][src]
                    s[x] = s[x][:keep].copy()

    def compare():
        for b in range(B):
            for c in range(Hkv):
                s, n = state[b][c], int(seq[b])
                assert pos[b, c, :n].tolist() == s["p"].tolist()
                at = [(int(table[b, i // page]), i % page) for i in range(n)]
                assert (np.stack([np64(cache.k[x, c, r]) for x, r in at]) == s["k"]).all()
                assert (np.stack([np64(cache.v[x, c, r]) for x, r in at]) == s["v"]).all()
                # lse of the attention is within 2^-18 sum|q||k| scale + 2^-20 (1 + |lse|) < 2^-12 here: so are the weights
                assert np.abs(np64(weight)[b, c, :n] - s["w"]).max() <= 2.0 ** -11 * s["w"].max()

    evict()
    compare()
    for step in range(4):
        q, kn, vn = (normal(g, (B, h, T, D), "bf16") for h in (Hq, Hkv, Hkv))
        drafts = [T, T - step]
        parent = np.stack([make_tree(g, T, "tree") for _ in range(B)])
        o, lse = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent), draft_len=ints(drafts))
        accepted = []
        for b in range(B):
            path = [t for t in range(drafts[b]) if True]
            leaf = path[int(torch.randint(0, len(path), (1,), generator=g))]
            line = [leaf]
            while parent[b][line[-1]] >= 0:
                line.append(int(parent[b][line[-1]]))
            accepted.append(line[::-1])
        path = np.full((B, T), -1)
        for b, a in enumerate(accepted):
            path[b, :len(a)] = a
        count = ints([len(a) for a in accepted])
        for b in range(B):
            for h in range(Hq):
                s = state[b][h // group]
                for t in range(drafts[b]):
                    line = [t]
                    while parent[b][line[-1]] >= 0:
                        line.append(int(parent[b][line[-1]]))
                    kk = np.concatenate([s["k"], np64(kn)[b, h // group, line]])
                    vv = np.concatenate([s["v"], np64(vn)[b, h // group, line]])
                    x = scale * (kk @ np64(q)[b, h, t])
                    m = x.max()
                    p = np.exp(x - m)
                    assert abs(float(lse[b, h, t]) - (m + np.log(p.sum()))) <= 2.0 ** -12
                    p /= p.sum()
                    tol = 2.0 ** -8 * np.abs(p @ vv) + (2.0 ** -8 + 2.0 ** -11) * (p @ np.abs(vv))
                    assert (np.abs(np64(o[b, h, t]) - p @ vv) <= tol).all()
        fa.cache_append(cache, kn.cuda(), vn.cuda(), path=ints(path), count=count, weight=weight, pos=pos, start=nxt)
        seq += count
        nxt += count
        fa.cache_weights(cache, q.cuda(), lse, weight, path=ints(path), count=count)
        for b, a in enumerate(accepted):
            for c in range(Hkv):
                s, n0 = state[b][c], len(state[b][c]["p"])
                s["k"] = np.concatenate([s["k"], np64(kn)[b, c, a]])
                s["v"] = np.concatenate([s["v"], np64(vn)[b, c, a]])
                s["w"] = np.concatenate([s["w"], np.zeros(len(a))])
                s["p"] = np.concatenate([s["p"], int(nxt[b]) - len(a) + np.arange(len(a))])
                for h in range(c * group, (c + 1) * group):
                    for i, t in enumerate(a):
                        see = n0 + i + 1
                        x = scale * (s["k"][:see] @ np64(q)[b, h, t])
                        s["w"][:see] += np.exp(x - x.max()) / np.exp(x - x.max()).sum()
        evict()
        compare()
    assert fa.fa_device_status() == (0, 0)


# ---------------------------------------------------------------- streams, graphs, threads

def small_case(fa, seed, lens=(300, 77), D=128, T=5, Hq=8, Hkv=2, page=16):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    k, v, table = make_pool(g, list(lens), Hkv, D, page, "bf16", room=T)
    cap = table.shape[1] * page
    c = dict(cache=fa.KVCache(k.cuda(), v.cuda(), ints(lens), table.cuda()), q=normal(g, (B, Hq, T, D), "bf16").cuda(),
             kn=normal(g, (B, Hkv, T, D), "bf16").cuda(), vn=normal(g, (B, Hkv, T, D), "bf16").cuda(),
             weight=torch.rand(B, Hkv, cap, generator=g).cuda(), pos=torch.arange(cap, dtype=torch.int32).expand(B, Hkv, cap).contiguous().cuda())
    all_four(fa, c)    # once: the eviction moves rows, the same ones every time, so that from now on a step repeats exactly
    return c


def all_four(fa, c, stream=None, **kw):
    """One step: attention, append, weights, eviction into separate buffers; its results."""
    cache = c["cache"]
    o, lse = fa.tree_attention(c["q"], c["kn"], c["vn"], cache, stream=stream)
    fa.cache_append(cache, c["kn"], c["vn"], stream=stream)
    out = torch.zeros_like(c["weight"])
    fa.cache_weights(cache, c["q"], lse, c["weight"], out=out, stream=stream)
    wo, po = torch.zeros_like(c["weight"]), torch.zeros_like(c["pos"])
    left = fa.cache_evict(cache, c["weight"], c["pos"], 60, weight_out=wo, pos_out=po, stream=stream)
    return [o, lse, out, wo, po, left]


def test_another_stream(fa):
    """Everything on a stream that is not the current one, named and entered, behind a long wait."""
    c = small_case(fa, 21)
    want = [t.clone() for t in all_four(fa, c)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for how in ("named", "handle", "entered"):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        if how == "entered":
            with torch.cuda.stream(s):
                got = all_four(fa, c)
        else:
            got = all_four(fa, c, stream=s if how == "named" else s.cuda_stream)
            # the current stream's allocations meanwhile must not meet the call's workspaces
            junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(8)]
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), how
        torch.cuda.synchronize()
    del junk


def test_a_named_stream_has_its_own_memory(fa):
    """A block that the current stream has freed, while work there is still to write it, must not be part of a call
    on another stream; nor may zeros be filled in by the current stream."""
    c = small_case(fa, 22)
    q, kn, vn, cache = c["q"], c["kn"], c["vn"], c["cache"]
    want = [t.clone() for t in fa.tree_attention(q, kn, vn, cache)]
    want.append(fa.cache_weights(cache, q, want[1]).clone())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sizes = sorted({fa.tree_workspace_bytes(q.shape[1], kn.shape[1], q.shape[2], q.shape[3]), fa.weights_workspace_bytes(),
                    q.nbytes, want[1].nbytes, want[2].nbytes})
    for how in (s, s.cuda_stream):
        torch.cuda._sleep(100_000_000)
        for size in sizes:          # written behind the wait, free for the current stream at once
            for _ in range(4):
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xff)
        o, lse = fa.tree_attention(q, kn, vn, cache, stream=how)
        w = fa.cache_weights(cache, q, want[1], stream=how)
        s.synchronize()
        torch.cuda.synchronize()
        for a, b in zip((o, lse, w), want):
            assert torch.equal(a, b)


def test_two_streams_at_once(fa):
    cs = [small_case(fa, 30 + i, lens=(900 + 50 * i, 400)) for i in range(2)]
    want = [[t.clone() for t in all_four(fa, c)] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = []
        for s, c in zip(streams, cs):
            with torch.cuda.stream(s):
                got.append(all_four(fa, c))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_threads_on_one_stream(fa):
    import threading
    cs = [small_case(fa, 40 + i, lens=(700, 300 + 80 * i)) for i in range(2)]
    want = [[t.clone() for t in all_four(fa, c)] for c in cs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(30):
            got = all_four(fa, cs[i])
            torch.cuda.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_captured_graphs_follow_the_lengths(fa):
    """Two graphs captured on one stream and replayed at once on two; lengths and tables change between replays."""
    cs = [small_case(fa, 50 + i, lens=(500, 200)) for i in range(2)]
    graphs, outs = [], []
    for c in cs:
        c["cache"].k.nan_to_num_(0, 0, 0), c["cache"].v.nan_to_num_(0, 0, 0)   # every page will be somebody's
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            torch.zeros(1000, device="cuda").zero_()          # a memset node before the first call
            out = all_four(fa, c)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in cs]
    for lens in ((500, 200), (0, 37), (129, 500), (16, 1)):
        want = []
        for c in cs:
            c["cache"].seq_len.copy_(ints(lens))
            c["cache"].table.copy_(c["cache"].table.flip(1))
        torch.cuda.synchronize()
        for c in cs:
            all_four(fa, c)                                     # once: its eviction moves rows, the same ones every time
            want.append([t.clone() for t in all_four(fa, c)])
        torch.cuda.synchronize()
        for out in outs:
            out[0].fill_(7), out[1].fill_(7)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            for a, b in zip(out, w):
                assert torch.equal(a, b), lens


def test_given_workspace(fa):
    c = small_case(fa, 60)
    want = [t.clone() for t in all_four(fa, c)]
    ws = torch.full((1 << 23,), 255, dtype=torch.uint8, device="cuda")       # NaN patterns: no initial value is needed
    o, lse = fa.tree_attention(c["q"], c["kn"], c["vn"], c["cache"], workspace=ws)
    ws.fill_(255)
    out = fa.cache_weights(c["cache"], c["q"], lse, c["weight"], out=torch.zeros_like(c["weight"]), workspace=ws)
    ws.fill_(255)
    wo = torch.zeros_like(c["weight"])
    fa.cache_evict(c["cache"], c["weight"], c["pos"], 60, weight_out=wo, pos_out=torch.zeros_like(c["pos"]), workspace=ws)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and torch.equal(out, want[2]) and torch.equal(wo, want[3])
    from programming_flashattention_fwd_gb300.binding import FaError
    with pytest.raises(FaError) as e:
        fa.tree_attention(c["q"], c["kn"], c["vn"], c["cache"], workspace=ws[:1024])
    assert e.value.status == 16


# ---------------------------------------------------------------- the edges of the sizes

def test_lengths_out_of_range_are_clamped(fa):
    c = small_case(fa, 70, lens=(64, 64), T=4, page=16)
    cache, cap = c["cache"], c["cache"].capacity
    results = []
    for lens in ([cap + 1000, -5], [cap, 0]):
        cache.seq_len.copy_(ints(lens))
        cache.k.nan_to_num_(0, 0, 0), cache.v.nan_to_num_(0, 0, 0)
        o, lse = fa.tree_attention(c["q"], c["kn"], c["vn"], cache, draft_len=ints([2000, 3]), o=torch.zeros_like(c["q"]))
        out = fa.cache_weights(cache, c["q"], lse, c["weight"], count=ints([99, -3]), path=ints([[0, 1, 2, 3]] * 2), out=torch.zeros_like(c["weight"]))
        results.append((o, lse[0], out))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert fa.fa_device_status() == (0, 0)


def test_many_sequences_with_weights(fa):
    """More sequences than one warp looks at in one go."""
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 400, 75)]
    run_weights(fa, "bf16", 2, 1, 64, lens, [min(n, 3 + i % 40) for i, n in enumerate(lens)], 50, 16)
    run_weights(fa, "bf16", 2, 1, 64, lens, [min(n, 3 + i % 140) for i, n in enumerate(lens)], 150, 16)


def test_weights_of_a_long_prompt(fa):
    """The variant for long prompts: its sums against the oracle's, with one head."""
    run_weights(fa, "bf16", 1, 1, 64, [4200], [4200], 4200, 128, poison=False)


def test_pool_of_more_than_32_bits(fa):
    """Pages at the far end of a pool of more than 2^32 elements."""
    g = torch.Generator().manual_seed(80)
    page, Hkv, D, n, T = 128, 2, 64, 300, 6
    num = (2 ** 32 + 2 ** 28) // (Hkv * page * D)
    k, v, table = make_pool(g, [n], Hkv, D, page, "bf16", room=T)
    far = torch.arange(num - table.shape[1], num)[None]
    K, V = (torch.empty(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K[far[0].cuda()], V[far[0].cuda()] = k[table[0].long()].cuda(), v[table[0].long()].cuda()
    q, kn, vn = (normal(g, (1, h, T, D), "bf16").cuda() for h in (4, Hkv, Hkv))
    caches = [fa.KVCache(k.cuda(), v.cuda(), ints([n]), table.cuda()), fa.KVCache(K, V, ints([n]), ints(far))]
    w0 = torch.rand(1, Hkv, caches[0].capacity, generator=g)
    results = []
    for c in caches:
        weight, pos = w0.cuda(), torch.arange(c.capacity, dtype=torch.int32).expand(1, Hkv, c.capacity).contiguous().cuda()
        o, lse = fa.tree_attention(q, kn, vn, c)
        fa.cache_append(c, kn, vn)
        c.seq_len.add_(T)
        fa.cache_weights(c, q, lse, weight)
        fa.cache_evict(c, weight, pos, 200)
        o2, lse2 = fa.tree_attention(q, kn, vn, c)
        results.append((o, lse, weight, pos, o2, lse2))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_evict_more_slots_than_fit_in_shared_memory(fa):
    """One head with more slots a CTA than keys are held for, and tables of more pages."""
    n, keep, page = 400_000, 150_000, 16
    g = torch.Generator().manual_seed(81)
    k = torch.zeros(-(-n // page), 1, page, 64, dtype=torch.bfloat16, device="cuda")
    k[:, 0, :, 0] = (torch.arange(n, device="cuda") % 251).reshape(-1, page).to(torch.bfloat16)
    v = k.clone()
    for kind in ("spread", "ties"):
        w = torch.rand(1, 1, k.shape[0] * page, generator=g) if kind == "spread" else torch.zeros(1, 1, k.shape[0] * page)
        pos = torch.arange(w.shape[2], dtype=torch.int32)[None, None]
        K, V, wd, pd = k.clone(), v.clone(), w.cuda(), pos.cuda()
        fa.cache_evict(fa.KVCache(K, V, ints([n])), wd, pd, keep, first=5, last=100, next_pos=ints([n]))
        dst, src = choose(w[0, 0].numpy(), pos[0, 0].numpy(), n, keep, 5, 100, n)
        pr = pos[0, 0].clone()
        pr[dst] = pr[src]
        assert torch.equal(pd[0, 0, :keep].cpu(), pr[:keep])
        assert torch.equal(K.reshape(-1, 64)[:keep, 0].cpu(), (pr[:keep] % 251).to(torch.bfloat16)) and torch.equal(K, V)
        assert torch.equal(wd[0, 0, :keep].cpu(), w[0, 0][pr[:keep].long()])


@pytest.mark.parametrize("D", [64, 256])
def test_tree_non_finite_marks_do_not_outlive_their_unit(fa, D):
    """Many units a CTA, some with non-finite drafted values: the others' rows are what they were."""
    g = torch.Generator().manual_seed(82)
    B, Hkv, T = 320, 2, 3
    k, v, table = make_pool(g, [10] * B, Hkv, D, 16, "bf16")
    q, kn, vn = (normal(g, (B, Hkv, T, D), "bf16") for _ in range(3))
    parent = np.tile(np.array([-1, 0, 0]), (B, 1))
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([10] * B), table.cuda())
    o1, l1 = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent))
    bad = torch.rand(B, generator=g) < 0.3
    vn[bad, :, 1, 5] = float("inf")
    o2, l2 = fa.tree_attention(q.cuda(), kn.cuda(), vn.cuda(), cache, parent=ints(parent))
    want = o1.clone()
    want[bad.cuda(), :, 1, 5] = float("inf")
    assert torch.equal(o2, want) and torch.equal(l1, l2)


# ---------------------------------------------------------------- waits that give up

def debug_call(fa, fn, cache, args, tail):
    from programming_flashattention_fwd_gb300 import cache as fc
    st = getattr(fc._library(), fn)(cache._c, *[None if a is None else a.data_ptr() for a in args], *tail)
    assert st == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 4), (128, 80), (256, 4)])
@pytest.mark.parametrize("inject", [1, 2])
def test_tree_waits_are_bounded(fa, D, Hq, inject):
    """A V tile that never comes: the call ends, the status says so, the rows concerned are NaN, the others right
    and the next call as well.  (Hq = 80: two row tiles side by side.)"""
    g = torch.Generator().manual_seed(90)
    B, Hkv, T, n = 40, 2, 4, 700
    k, v, table = make_pool(g, [n] * B, Hkv, D, 16, "bf16")
    q, kn, vn = (normal(g, (B, h, T, D), "bf16").cuda() for h in (Hq, Hkv, Hkv))
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([n] * B), table.cuda())
    want = fa.tree_attention(q, kn, vn, cache)
    o, lse = torch.zeros_like(q), torch.zeros(B, Hq, T, device="cuda")
    size = fa.tree_workspace_bytes(Hq, Hkv, T, D)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    debug_call(fa, "fa_tree_debug", cache, (q, kn, vn, None, None, o, lse),
               (Hq, T, D ** -0.5, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream, 3_000_000, inject))
    st, word = fa.fa_device_status()
    assert st == 12 and word & 1
    gone = torch.isnan(lse)
    assert gone.any() and torch.equal(torch.isnan(o).all(3), gone) and torch.equal(torch.isnan(o).any(3), gone)
    assert torch.equal(o[~gone], want[0][~gone]) and torch.equal(lse[~gone], want[1][~gone])
    if inject == 1:
        assert gone.all()
    else:
        heads = gone.reshape(B, Hkv, -1)                  # CTA 0 has the first units; what it shares goes with it
        assert heads[0, 0].any() and not heads[-1].any()
    assert fa.fa_device_status() == (0, 0)
    again = fa.tree_attention(q, kn, vn, cache)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1]) and fa.fa_device_status() == (0, 0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,with_path", [(6, True), (40, False), (300, False)])
@pytest.mark.parametrize("inject", [1, 2])
def test_weights_waits_are_bounded(fa, D, T, with_path, inject):
    g = torch.Generator().manual_seed(91)
    B, Hq, Hkv, n = 24, 4, 2, 1100
    k, v, table = make_pool(g, [n] * B, Hkv, D, 16, "bf16")
    q, lse = normal(g, (B, Hq, T, D), "bf16").cuda(), torch.randn(B, Hq, T, generator=g).cuda() + 4
    cache = fa.KVCache(k.cuda(), v.cuda(), ints([n] * B), table.cuda())
    path, count = (ints([list(range(T))] * B), ints([T] * B)) if with_path else (None, None)
    want = fa.cache_weights(cache, q, lse, path=path, count=count)
    out = torch.zeros_like(want)
    size = fa.weights_workspace_bytes()
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    debug_call(fa, "fa_weights_debug", cache, (q, lse, path, count, None, out),
               (Hq, T, 1, D ** -0.5, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream, 3_000_000, inject))
    st, word = fa.fa_device_status()
    assert st == 12 and word & 1
    used = torch.arange(cache.capacity, device="cuda") < n
    gone = torch.isnan(out)
    assert gone.any() and not gone[..., ~used].any()
    assert torch.equal(out[~gone], want[~gone])
    if inject == 1:
        assert gone[..., used].all()
    else:
        assert gone[0, 0].any() and not gone[-1].any()
    assert torch.equal(fa.cache_weights(cache, q, lse, path=path, count=count), want) and fa.fa_device_status() == (0, 0)
