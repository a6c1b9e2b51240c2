"""The backward pass without a GPU: its schedule (walked on the host), and the calls that it refuses."""
import math
import os
import shutil
import subprocess

import pytest
import torch

from programming_flashattention_fwd_gb300 import build as fa_build
from test_schedule_cpu import CSRC, ROOT, cuda_include


def test_schedule(tmp_path):
    cxx, inc = shutil.which("g++") or shutil.which("c++"), cuda_include()
    if not cxx or not inc:
        pytest.skip("needs a host C++ compiler and the CUDA headers")
    exe = str(tmp_path / "bwd_schedule_check")
    r = subprocess.run([cxx, "-std=c++17", "-O2", f"-I{CSRC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{inc}",
                        os.path.join(ROOT, "tests", "bwd_schedule_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    from programming_flashattention_fwd_gb300 import grad
    return grad._library()


# Addresses that validation never reads: 16-byte aligned and apart.
A = {n: (i + 1) << 32 for i, n in enumerate(("q", "k", "v", "o", "lse", "d_o", "dlse", "dq", "dk", "dv", "ws"))}
GOOD = dict(A, B=1, Hq=4, Hkv=2, Sq=200, Sk=300, D=128, causal=1, scale=0.125, dtype=0, size=1 << 40)


def call(lib, **over):
    a = dict(GOOD, **over)
    return lib.fa_bwd(*(a[x] for x in ("q", "k", "v", "o", "lse", "d_o", "dlse", "dq", "dk", "dv", "B", "Hq", "Hkv", "Sq", "Sk", "D", "causal", "scale", "dtype",
                                        "ws", "size")), None)


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), 2), (dict(Sq=-5), 2), (dict(Sk=-1), 2), (dict(Sk=0), 2), (dict(Sq=2 ** 31 - 1), 2), (dict(Sk=2 ** 31 - 1), 2),
    (dict(B=100000, Hq=100000, Hkv=1), 2), (dict(Hq=0), 3), (dict(Hkv=0), 3), (dict(Hq=6, Hkv=4), 3), (dict(D=96), 4), (dict(D=32), 4),
    (dict(causal=3), 13), (dict(causal=-1), 13), (dict(dtype=2), 15), (dict(scale=math.nan), 7), (dict(scale=math.inf), 7), (dict(scale=3e38), 7),
    (dict(size=0), 16), (dict(ws=None), 1), (dict(ws=A["ws"] + 16), 5),
    *[({n: None}, 1) for n in ("q", "k", "v", "o", "lse", "d_o", "dk", "dv")],
    *[({n: A[n] + 8}, 5) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")], (dict(lse=A["lse"] + 2), 5), (dict(dlse=A["dlse"] + 2), 5),
    *[({n: A[m] + 16}, 6) for n in ("dq", "dk", "dv") for m in ("q", "k", "v", "o", "d_o", "lse", "dlse", "ws") if n != m], (dict(dk=A["dv"]), 6), (dict(dq=A["dk"]), 6),
    (dict(ws=A["q"] + 64), 6),
])
def test_refusals(lib, over, code):
    assert call(lib, **over) == code


def test_nothing_to_do(lib):
    assert call(lib, B=0) == 0
    assert call(lib, Sq=0, Sk=0) == 0
    assert call(lib, dq=None, dk=None, dv=None) == 0


def test_workspace_bytes(lib):
    """Two padded vectors; parts where whole units would leave SMs idle, at most two of a CTA for a result."""
    f = lib.fa_bwd_workspace_bytes
    assert f(1, 38, 38, 512, 512, 128, 0) == 2 * 38 * 512 * 4   # 152 units as long as each other
    assert f(1, 32, 8, 100, 100, 96, 0) == 0 and f(0, 4, 2, 100, 100, 64, 0) == 0 and f(1, 3, 2, 100, 100, 64, 0) == 0 and f(1, 4, 2, 100, 100, 64, 3) == 0
    for args in ((1, 1, 1, 1, 100000, 64), (1, 32, 1, 4096, 4096, 128), (1, 2, 2, 128, 128, 64), (3, 5, 5, 700, 64, 256)):
        B, Hq, Hkv, Sq, Sk, D = args
        for causal in (0, 1, 2):
            assert f(*args, causal) - 2 * B * Hq * -(-Sq // 128) * 128 * 4 in range(0, 3 * 2 * 152 * 128 * D * 4 + 1), args


def test_binding_refuses():
    """What the binding turns down before it reaches the library."""
    import programming_flashattention_fwd_gb300 as fa
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_bwd(x, x, x, x, lse, x)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        fa.attention_bwd(x.float(), x, x, x, lse, x)
    with pytest.raises(ValueError, match="4-D"):
        fa.attention_bwd(x[0], x, x, x, lse, x)
