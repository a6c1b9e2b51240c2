"""GPU tests of attention's backward pass against its formulas in float64.

Tolerances, from the arithmetic.  u = eps / 2 is the type's rounding (2^-8 bf16, 2^-11 fp16).  First-order terms, doubled where
they are products of two:

  p     a score is an fp32 sum of exact products of up to 256 terms: e = 2^-18 scale sum |q||k|; the exponent's own roundings
        2^-22 (1 + |lse|) and the hardware exponential 2^-21:  |dp| <= p rho,  rho = e + 2^-22 (1 + |lse|) + 2^-21.
        For the sums of dv it is rounded to the type once more (u); fp16 values are held 2^12 times as large, so that only
        those below 2^-26 have an absolute error, 2^-37.
  dv    |ddv_j| <= sum_i (p_ij (2 rho + u) + f) |do_i| + 2^-18 sum_i p_ij |do_i| + u |dv_j|,  f = 2^-37 in fp16, 0 in bf16
  ds    do.v has an error of 2^-18 sum |do||v|, delta of 2^-18 sum |do||o| + 2^-23 |dlse|; ds is rounded to the type (u; in fp16
        half a step of 2^-25 at least):  |dds| <= |ds| (2 rho + u) + p (2^-18 (sum |do||v| + sum |do||o|) + 2^-23 |dlse|) + (2^-25)
  dq    |ddq_i| <= |scale| (sum_j |dds_ij| |k_j| + 2^-18 sum_j |ds_ij| |k_j|) + u |dq_i|;  dk the same with q.
  Results below the type's normal range are off by half its smallest step at most: 2^-25 in fp16, 2^-134 in bf16.
  A probability below fp32's normal range, 2^-126, is flushed to zero (ex2.approx.ftz): its error is up to 2^-126 itself, that of ds
  2^-126 |do.v - delta|, and that of a bf16 ds below the normal range 2^-134.
"""
import pytest
import torch

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


def shut_of(Sq, Sk, causal):
    i, j = torch.arange(Sq, device="cuda")[:, None], torch.arange(Sk, device="cuda")
    return j > i + (Sk - Sq if causal == 2 else 0) if causal else torch.zeros(Sq, Sk, dtype=torch.bool, device="cuda")


def make(seed, B, Hq, Hkv, Sq, Sk, D, dtype, causal, std=1.0, dlse=False, scale=None):
    """Inputs on the GPU, with o and lse of the forward pass from float64, rounded."""
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(DT[dtype])  # noqa: E731
    c = dict(q=n(B, Hq, Sq, D, std=std), k=n(B, Hkv, Sk, D, std=std), v=n(B, Hkv, Sk, D), do=n(B, Hq, Sq, D), causal=causal,
             scale=D ** -0.5 if scale is None else scale, dlse=torch.randn(B, Hq, Sq, generator=g, device="cuda") if dlse else None)
    k, v = (c[x].double().repeat_interleave(Hq // Hkv, 1) for x in "kv")
    s = (c["q"].double() @ k.transpose(2, 3) * c["scale"]).masked_fill(shut_of(Sq, Sk, causal), -float("inf"))
    lse = torch.logsumexp(s, 3)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    c["o"], c["lse"] = (p @ v).to(DT[dtype]), lse.float()
    return c


def want(c, dtype):
    """(dq, dk, dv) in float64 and how far each may be off."""
    q, k, v, o, do, lse = (c[x].double() for x in ("q", "k", "v", "o", "do", "lse"))
    B, Hq, Sq, D = q.shape
    Hkv, Sk = k.shape[1:3]
    G, u, scale = Hq // Hkv, U[dtype], c["scale"]
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    shut = shut_of(Sq, Sk, c["causal"])
    tiny = 1.0 if dtype == "fp16" else 0.0
    p = torch.exp(q @ kk.transpose(2, 3) * scale - lse[..., None]).masked_fill(shut, 0.0)
    e = 2.0 ** -18 * abs(scale) * (q.abs() @ kk.abs().transpose(2, 3))
    safe = torch.where(torch.isinf(lse), 0.0, lse)[..., None].abs()
    rho = e + 2.0 ** -22 * (1 + safe) + 2.0 ** -21
    dl = torch.zeros_like(lse) if c["dlse"] is None else c["dlse"].double()
    ds = p * (do @ vv.transpose(2, 3) - ((do * o).sum(3) - dl)[..., None])
    a = 2.0 ** -18 * (do.abs() @ vv.abs().transpose(2, 3) + (do.abs() * o.abs()).sum(3)[..., None]) + 2.0 ** -23 * dl.abs()[..., None]
    seen = (~shut).double()
    dp = (do @ vv.transpose(2, 3) - ((do * o).sum(3) - dl)[..., None]).abs()
    far = 2.0 ** -126 * (dp + 1) * seen + ds.abs() * (2 * rho + u) + p * a + tiny * 2.0 ** -25 * seen + 2.0 ** -18 * ds.abs()
    fold = lambda x: x.reshape(B, Hkv, G, Sk, D).sum(2)  # noqa: E731
    t = lambda x: x.transpose(2, 3)  # noqa: E731
    dq, dk, dv = scale * (ds @ kk), fold(scale * (t(ds) @ q)), fold(t(p) @ do)
    low = max(tiny * 2.0 ** -25, 2.0 ** -134)
    tq = abs(scale) * (far @ kk.abs()) + u * dq.abs() + low
    tk = fold(abs(scale) * (t(far) @ q.abs())) + u * dk.abs() + low
    tv = fold(t(p * (2 * rho + u + 2.0 ** -18) + (tiny * 2.0 ** -37 + 2.0 ** -126) * seen) @ do.abs()) + u * dv.abs() + low
    return (dq, dk, dv), (tq, tk, tv)


def run(fa, c, **over):
    return fa.attention_bwd(c["q"], c["k"], c["v"], c["o"], c["lse"], c["do"], causal=c["causal"], scale=c["scale"], dlse=c["dlse"], **over)


def near(got, c, dtype):
    ref, tol = want(c, dtype)
    for name, x, y, t in zip(("dq", "dk", "dv"), got, ref, tol):
        d = (x.double() - y).abs()
        assert torch.isfinite(x.double()).all(), f"{name} is not finite at {torch.nonzero(~torch.isfinite(x.double()))[0].tolist()}"
        bad = torch.nonzero(d > t)
        assert len(bad) == 0, f"{name} off by {d[tuple(bad[0])]:.3g} (may be {t[tuple(bad[0])]:.3g}) at {bad[0].tolist()}, {len(bad)} places of {d.numel()}"


# one tile, one step; ragged; several tiles and steps; shared heads; each head dimension, type and mask
SHAPES = [
    (1, 1, 1, 128, 128, 64), (1, 1, 1, 128, 128, 128), (1, 1, 1, 128, 128, 256),
    (1, 2, 1, 1, 1, 64), (2, 2, 2, 1, 300, 128), (1, 2, 2, 300, 1, 128), (1, 1, 1, 5, 7, 256),
    (2, 4, 2, 200, 333, 64), (1, 6, 2, 257, 129, 128), (2, 2, 1, 190, 260, 256), (1, 7, 1, 130, 500, 64),
    (3, 5, 5, 127, 255, 128), (1, 4, 4, 640, 640, 64), (1, 8, 2, 520, 776, 128), (1, 4, 2, 385, 449, 256),
]


@pytest.mark.parametrize("causal", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(fa, shape, dtype, causal):
    c = make(sum(shape) + causal, *shape, dtype, causal, dlse=sum(shape) % 2 == 0)
    near(run(fa, c), c, dtype)
    assert fa.fa_device_status()[0] == 0


# more units than SMs, whole (not cut) units of many steps, several rounds of a CTA
@pytest.mark.parametrize("shape,dtype,causal", [
    ((2, 12, 6, 1100, 1500, 128), "bf16", 1), ((2, 12, 12, 1500, 1100, 64), "bf16", 2), ((2, 8, 4, 1300, 1300, 256), "bf16", 1),
    ((4, 16, 8, 500, 700, 128), "fp16", 0), ((3, 20, 4, 515, 900, 64), "fp16", 1), ((2, 12, 12, 770, 770, 256), "fp16", 2),
], ids=str)
def test_several_rounds(fa, shape, dtype, causal):
    c = make(11, *shape, dtype, causal)
    near(run(fa, c), c, dtype)


# few units of many steps: their steps are cut, and the parts joined
@pytest.mark.parametrize("shape,dtype,causal", [
    ((1, 2, 2, 130, 9000, 64), "bf16", 2), ((1, 8, 1, 1024, 1024, 128), "bf16", 1), ((1, 14, 1, 600, 2000, 128), "fp16", 2), ((1, 2, 1, 100, 3000, 256), "bf16", 0),
    ((1, 8, 1, 700, 700, 256), "fp16", 1), ((1, 16, 1, 900, 64, 64), "bf16", 0), ((1, 8, 1, 3000, 700, 128), "bf16", 2), ((1, 8, 2, 1500, 4000, 64), "bf16", 1),
], ids=str)
def test_cut_units(fa, shape, dtype, causal):
    c = make(12, *shape, dtype, causal, dlse=True)
    assert fa.bwd_workspace_bytes(*shape, causal) > 2 * shape[0] * shape[1] * -(-shape[3] // 128) * 128 * 4
    full = [torch.full_like(c[x], float("nan")) for x in "qkv"]
    got = run(fa, c, dq=full[0], dk=full[1], dv=full[2])
    near(got, c, dtype)
    again = run(fa, c)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("scale", [0.0, -0.125, 0.9])
def test_scales(fa, scale):
    """Negative and zero scales, as the forward pass takes them, and large logits."""
    c = make(5, 1, 4, 2, 200, 300, 64, "bf16", 1, std=2.0 if scale > 0 else 1.0, scale=scale)
    near(run(fa, c), c, "bf16")


def test_rows_that_see_nothing(fa):
    """Bottom-right with more queries than keys: the first rows see nothing; lse = -inf, o = 0, dq = 0."""
    for D in (64, 128, 256):
        c = make(6, 1, 2, 1, 500, 140, D, "bf16", 2)
        dq, dk, dv = run(fa, c)
        near((dq, dk, dv), c, "bf16")
        assert torch.isinf(c["lse"][:, :, :360]).all() and (dq[:, :, :360] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_gradient_of_an_empty_row_s_lse(fa, D):
    """A row that sees nothing has lse = -inf, whose gradient is often NaN or infinite (that of exp(lse - m), say): it has no effect."""
    c = make(27, 1, 2, 1, 200, 90, D, "bf16", 2, dlse=True)
    empty = torch.isinf(c["lse"])
    assert empty.sum() == 2 * 110
    plain = run(fa, c)
    near(plain, c, "bf16")
    for x in (float("nan"), float("inf"), -float("inf")):
        c["dlse"] = c["dlse"].masked_fill(empty, x)
        assert all(torch.equal(a, b) for a, b in zip(run(fa, c), plain))


def test_keys_that_nobody_sees(fa):
    """Top-left with more keys than queries: dk and dv of the keys behind are zero, whatever was there."""
    for D in (64, 128, 256):
        c = make(7, 1, 2, 2, 70, 500, D, "fp16", 1)
        full = [torch.full_like(x, float("nan")) for x in (c["q"], c["k"], c["v"])]
        got = run(fa, c, dq=full[0], dk=full[1], dv=full[2])
        assert all(x is y for x, y in zip(got, full))
        near(got, c, "fp16")
        assert (got[1][:, :, 70:] == 0).all() and (got[2][:, :, 70:] == 0).all()


def test_no_queries(fa):
    """Sq = 0: dk and dv are zeros."""
    z = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dq, dk, dv = fa.attention_bwd(z(2, 4, 0, 64), z(2, 2, 9, 64), z(2, 2, 9, 64), z(2, 4, 0, 64), torch.ones(2, 4, 0, device="cuda"), z(2, 4, 0, 64),
                                  dk=z(2, 2, 9, 64), dv=z(2, 2, 9, 64))
    assert dq.shape == (2, 4, 0, 64) and (dk == 0).all() and (dv == 0).all()


def test_parts_of_the_results(fa):
    """dq alone, dk and dv alone: the same bits as together; nothing else is returned."""
    for shape in ((1, 4, 2, 200, 333, 64), (1, 8, 1, 1024, 1024, 128)):
        c = make(13, *shape, "bf16", 1)
        dq, dk, dv = run(fa, c)
        a, b = run(fa, c, need_kv=False), run(fa, c, need_q=False)
        near((a[0], b[1], b[2]), c, "bf16")
        assert a[1] is None and a[2] is None and b[0] is None
        assert run(fa, c, need_q=False, need_kv=False) == (None, None, None)
        if shape[1] == 4:   # not cut, so the order of the sums is the same
            assert torch.equal(a[0], dq) and torch.equal(b[1], dk) and torch.equal(b[2], dv)


def test_alignment(fa):
    """Tensors on 16 bytes but not on 32."""
    for D in (64, 128, 256):
        c = make(14, 1, 2, 1, 150, 170, D, "bf16", 1)
        want_ = run(fa, c)

        def off(x):
            flat = torch.zeros(x.numel() + 8, dtype=x.dtype, device="cuda")
            y = flat[8:].view(x.shape)
            assert y.data_ptr() % 32 == 16
            return y.copy_(x)
        moved = dict(c, **{n: off(c[n]) for n in ("q", "k", "v", "o", "do")})
        got = run(fa, moved, dq=off(c["q"]), dk=off(c["k"]), dv=off(c["v"]))
        assert all(torch.equal(x, y) for x, y in zip(got, want_))


def test_streams_graphs_and_workspaces(fa):
    """A call on a stream of its own; calls on two streams at once; two graphs with calls that are cut (parts in a workspace of the graph's own),
    replayed at once over new inputs."""
    c = make(15, 1, 8, 1, 1024, 1024, 128, "bf16", 1)
    d = make(16, 1, 8, 1, 1024, 1024, 128, "bf16", 1)
    wc, wd = run(fa, c), run(fa, d)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(run(fa, c, stream=s1), run(fa, d, stream=s2)) for _ in range(4)]
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(a, b) for a, b in zip(x + y, wc + wd))
    graphs = []
    for t in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(fa, t)
        graphs.append((g, out))
    for x in ("q", "k", "v", "o", "do", "lse"):   # the other's inputs
        a = c[x].clone()
        c[x].copy_(d[x])
        d[x].copy_(a)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1] + graphs[1][1], wd + wc))


def test_given_workspace(fa):
    c = make(17, 1, 8, 1, 1024, 1024, 128, "bf16", 1)
    n = fa.bwd_workspace_bytes(1, 8, 1, 1024, 1024, 128, True)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")   # NaN, whatever it is read as
    got = run(fa, c, workspace=ws[:n])
    assert all(torch.equal(a, b) for a, b in zip(got, run(fa, c))) and (ws[n:] == 255).all()
    with pytest.raises(fa.FaError):
        run(fa, c, workspace=ws[:n - 32])


def test_more_than_32_bits_of_elements(fa):
    """65792 head planes of 256 x 128 elements: 2.2e9 in each tensor; the last sequence is as it is alone."""
    B, H, S, D = 257 * 8, 32, 256, 128
    g = torch.Generator("cuda").manual_seed(0)
    t = {x: torch.empty(B, H, S, D, dtype=torch.bfloat16, device="cuda") for x in ("q", "k", "v", "do")}
    assert t["q"].numel() > 2 ** 31
    for x in t.values():
        x[:-1] = 0.25
        x[-1] = torch.randn(H, S, D, generator=g, device="cuda")
    o, lse = fa.attention(t["q"], t["k"], t["v"], causal=True)
    got = fa.attention_bwd(t["q"], t["k"], t["v"], o, lse, t["do"], causal=True)
    one = {x: y[-1:].clone() for x, y in t.items()}
    alone = fa.attention_bwd(one["q"], one["k"], one["v"], o[-1:].clone(), lse[-1:].clone(), one["do"], causal=True)
    assert all(torch.equal(x[-1:], y) for x, y in zip(got, alone))
    c = dict(one, o=o[-1:].clone(), lse=lse[-1:].clone(), dlse=None, causal=1, scale=D ** -0.5)
    near(alone, c, "bf16")


def test_against_differences(fa):
    """Along random directions the gradients' products are the loss's differences: L = sum(do o) + sum(dlse lse) in float64.

    Tolerance: the tests' own (sum of its places times |direction|), that of o and lse, which the call takes rounded to the type
    (in `want`, delta is of the rounded o too: its error u sum |do||o| reaches ds times p), and the differences' own:
    step h = 1e-4 leaves h^2 / 6 of the third derivative and 1e-16 / h of rounding, together under 1e-6 of the sums here."""
    shape, dtype = (1, 4, 2, 90, 110, 64), "bf16"
    c = make(18, *shape, dtype, 2, dlse=True)
    got = run(fa, c)
    _, tol = want(c, dtype)
    B, Hq, Hkv, Sq, Sk, D = shape
    shut = shut_of(Sq, Sk, 2)

    def loss(q, k, v):
        kk, vv = k.repeat_interleave(Hq // Hkv, 1), v.repeat_interleave(Hq // Hkv, 1)
        s = (q @ kk.transpose(2, 3) * c["scale"]).masked_fill(shut, -float("inf"))
        return (torch.softmax(s, 3) @ vv * c["do"].double()).sum() + (torch.logsumexp(s, 3) * c["dlse"].double()).sum()
    x = [c[n].double() for n in "qkv"]
    # what the rounding of o does to ds: p u sum |do||o|, then through k and q
    kk = x[1].repeat_interleave(Hq // Hkv, 1)
    s = (x[0] @ kk.transpose(2, 3) * c["scale"]).masked_fill(shut, -float("inf"))
    e = torch.softmax(s, 3) * (U[dtype] * (c["do"].double().abs() * c["o"].double().abs()).sum(3))[..., None]
    extra = [c["scale"] * (e @ kk.abs()), (c["scale"] * (e.transpose(2, 3) @ x[0].abs())).reshape(B, Hkv, -1, Sk, D).sum(2), torch.zeros_like(x[2])]
    g = torch.Generator("cuda").manual_seed(5)
    for i in range(3):
        d = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        ends = [loss(*(y + sign * h * d if j == i else y for j, y in enumerate(x))) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        far = ((tol[i] + extra[i]) * d.abs()).sum() + 1e-6 * (got[i].double().abs() * d.abs()).sum()
        assert (slope - (got[i].double() * d).sum()).abs() <= far


def test_autograd(fa):
    """attention_ad's gradients are attention_bwd's, also through lse alone and for some of the inputs; a second order is refused."""
    g = torch.Generator("cuda").manual_seed(19)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, do, dlse = n(2, 4, 70, 64), n(2, 2, 90, 64), n(2, 2, 90, 64), n(2, 4, 70, 64), torch.randn(2, 4, 70, generator=g, device="cuda")
    o, lse = fa.attention(q, k, v, causal="bottom_right", scale=0.2)

    def leaves(*need):
        return [x.clone().requires_grad_(y) for x, y in zip((q, k, v), need)]
    a = leaves(True, True, True)
    ao, alse = fa.attention_ad(*a, causal="bottom_right", scale=0.2)
    assert torch.equal(ao, o) and torch.equal(alse, lse)
    torch.autograd.backward((ao, alse), (do, dlse))
    want_ = fa.attention_bwd(q, k, v, o, lse, do, causal=2, scale=0.2, dlse=dlse)
    assert all(torch.equal(x.grad, y) for x, y in zip(a, want_))
    a = leaves(True, False, False)
    fa.attention_ad(*a, causal=2, scale=0.2)[1].sum().backward()   # lse alone; its gradient is an expanded one
    want_ = fa.attention_bwd(q, k, v, o, lse, torch.zeros_like(o), causal=2, scale=0.2, dlse=torch.ones_like(lse), need_kv=False)
    assert torch.equal(a[0].grad, want_[0]) and a[1].grad is None and a[2].grad is None
    a = leaves(False, False, True)
    x, _ = fa.attention_ad(*a, causal=2, scale=0.2)
    x.transpose(1, 2).backward(do.transpose(1, 2))   # a gradient with other strides
    want_ = fa.attention_bwd(q, k, v, o, lse, do, causal=2, scale=0.2, need_q=False)
    assert torch.equal(a[2].grad, want_[2]) and a[0].grad is None and a[1].grad is None
    a = leaves(True, True, True)
    x = torch.autograd.grad(fa.attention_ad(*a)[0].float().pow(2).sum(), a, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        x.sum().backward()


def test_autograd_is_not_captured(fa):
    """attention_ad and rotary_ad refuse a capture whose gradients would be captured too; without gradients they are captured."""
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    leaf, table = q.clone().requires_grad_(), fa.RotaryTable(64)
    fa.attention_ad(q, q, q), fa.rotary_ad(table, q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for bad in (lambda: fa.attention_ad(leaf, q, q), lambda: fa.rotary_ad(table, leaf)):
            with pytest.raises(RuntimeError, match="captured"):
                bad()
        fa.attention_ad(q, q, q), fa.rotary_ad(table, q)
    g.replay()
    torch.cuda.synchronize()


def test_a_backward_pass_is_not_captured(fa):
    """Nor is the backward of a call that was made before the capture, on the same stream; the call's graph serves afterwards."""
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    q, table = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device="cuda"), fa.RotaryTable(64)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        leaves = [q.clone().requires_grad_() for _ in range(2)]
        outs, do = (fa.attention_ad(leaves[0], q, q)[0], fa.rotary_ad(table, leaves[1])), torch.ones_like(q)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        for o, x in zip(outs, leaves):
            with pytest.raises(RuntimeError, match="captured"):
                torch.autograd.grad(o, x, do, retain_graph=True)
        fa.attention(q, q, q)
    g.replay()
    with torch.cuda.stream(s):
        for o, x in zip(outs, leaves):
            o.backward(do)
            assert x.grad is not None
    torch.cuda.synchronize()


def test_a_layer_s_gradients(fa):
    """Projection, rotation, attention and their gradients as a training step runs them, against float64 autograd over the same
    products.  Tolerance: every tensor between is rounded to the type, and what comes out has passed seven such roundings
    (rotated q and k, o, P, dS, the gradients of rotated q and k, and the results): in the 2-norm each adds u / sqrt(3) of its
    own size at most, and the Jacobians between scale these like the values themselves; 16 u in all leaves a factor of 4."""
    B, T, Hq, Hkv, D = 2, 150, 4, 2, 64
    g = torch.Generator("cuda").manual_seed(21)
    x = torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
    do = torch.randn(B, Hq, T, D, generator=g, device="cuda").to(torch.bfloat16)
    table = fa.RotaryTable(D, rot=32, interleaved=True)
    split = lambda y: (y.view(B, T, -1, D).transpose(1, 2)[:, :Hq], y.view(B, T, -1, D).transpose(1, 2)[:, Hq:Hq + Hkv],  # noqa: E731
                       y.view(B, T, -1, D).transpose(1, 2)[:, Hq + Hkv:])
    leaf = x.clone().requires_grad_()
    q, k, v = split(leaf)
    q, k = fa.rotary_ad(table, q, k)
    fa.attention_ad(q, k, v.contiguous(), causal=True)[0].backward(do)
    ref = x.double().requires_grad_()
    q, k, v = split(ref)
    t = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(table.frequencies, device="cuda", dtype=torch.float64)

    def turn(y):
        a, b = y[..., 0:32:2], y[..., 1:32:2]
        pair = torch.stack((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()), -1).flatten(-2)
        return torch.cat((pair, y[..., 32:]), -1)
    q, k = turn(q), turn(k).repeat_interleave(Hq // Hkv, 1)
    s = (q @ k.transpose(2, 3) * D ** -0.5).masked_fill(shut_of(T, T, 1), -float("inf"))
    (torch.softmax(s, 3) @ v.repeat_interleave(Hq // Hkv, 1)).backward(do.double())
    for a, b in zip(split(leaf.grad.double()), split(ref.grad)):
        assert (a - b).norm() <= 16 * U["bf16"] * b.norm()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out(fa, D):
    """Every CTA leaves out its first load of v or d_o: the call ends, reports it, and leaves NaN in every row; the next is whole."""
    from programming_flashattention_fwd_gb300 import grad
    for shape in ((2, 4, 2, 300, 300, D), (1, 8, 1, 1024, 1024, D)):   # whole units, cut ones
        c = make(22, *shape, "bf16", 1)
        out = [torch.zeros_like(c[x]) for x in "qkv"]
        n = fa.bwd_workspace_bytes(*shape, 1)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        B, Hq, Hkv, Sq, Sk, _ = shape
        st = grad._library().fa_bwd_debug(*(c[x].data_ptr() for x in ("q", "k", "v", "o", "lse", "do")), None, *(x.data_ptr() for x in out), B, Hq, Hkv, Sq, Sk, D, 1,
                                          c["scale"], 0, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream, 2_000_000, 1)
        assert st == 0
        status, word = fa.fa_device_status()
        assert status == 12 and word & 1
        assert all(torch.isnan(x).all() for x in out)
        assert fa.fa_device_status()[0] == 0
        near(run(fa, c), c, "bf16")
        assert fa.fa_device_status()[0] == 0


def test_a_wait_for_a_long_unit(fa):
    """Units of 8192 steps (more than 8 ms) under a limit of 4 ms, which is for a step or two: the wait for a whole unit has more."""
    from programming_flashattention_fwd_gb300 import grad
    B, Hq, Hkv, Sq, Sk, D = shape = 1, 160, 1, 1, 8192 * 64, 256
    g = torch.Generator("cuda").manual_seed(28)
    q, o, do, k, v = (torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16) for s in [(B, Hq, Sq, D)] * 3 + [(B, Hkv, Sk, D)] * 2)
    lse = torch.full((B, Hq, Sq), 13.0, device="cuda")
    want_, _, _ = fa.attention_bwd(q, k, v, o, lse, do, need_kv=False)
    dq = torch.zeros_like(q)
    ws = torch.zeros(fa.bwd_workspace_bytes(*shape), dtype=torch.uint8, device="cuda")
    st = grad._library().fa_bwd_debug(*(x.data_ptr() for x in (q, k, v, o, lse, do)), None, dq.data_ptr(), None, None, *shape, 0, D ** -0.5, 0, ws.data_ptr(),
                                      ws.nbytes, torch.cuda.current_stream().cuda_stream, 4_000_000, 0)
    assert st == 0 and fa.fa_device_status()[0] == 0
    assert torch.isfinite(dq.float()).all() and torch.equal(dq, want_)
