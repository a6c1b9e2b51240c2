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
"""
import numpy as np
import pytest
import torch

from cache_oracle import attend
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
