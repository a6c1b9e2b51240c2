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


def test_keys_that_nobody_sees(fa):
    """Top-left with more keys than queries: dk and dv of the keys behind are zero, whatever was there."""
    for D in (64, 128, 256):
        c = make(7, 1, 2, 2, 70, 500, D, "fp16", 1)
        full = [torch.full_like(x, float("nan")) for x in (c["q"], c["k"], c["v"])]
        got = run(fa, c, dq=full[0], dk=full[1], dv=full[2])
        assert all(x is y for x, y in zip(got, full))
        near(got, c, "fp16")
        assert (got[1][:, :, 70:] == 0).all() and (got[2][:, :, 70:] == 0).all()
