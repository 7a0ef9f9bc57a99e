"""Workspaces of exactly the stated sizes: what they held before does not enter
the results, and nothing beside them is written."""
import pytest

import fp32_blocked_gemm_amd as og
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
CODES = {"float32": og.F32, "bfloat16": og.BF16}


def held(size, byte):
    """(all, the workspace inside it)."""
    t = torch()
    whole = t.full((size + 8192,), byte, dtype=t.uint8, device="cuda")
    return whole, whole[4096:4096 + size]


def untouched(whole, size, byte):
    return bool((whole[:4096] == byte).all() and (whole[4096 + size:] == byte).all())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,v,d", [(1, 1, 1), (3, 70, 33), (8, 1000, 96), (9, 1000, 96), (300, 777, 130),
                                   (1000, 5000, 40), (5000, 9001, 24), (40, 9001, 8200)])
def test_cross_entropy(n, v, d, dtype):
    t = torch()
    gen = t.Generator().manual_seed(n + v)
    kind = getattr(t, dtype)
    x = t.randn((n, d), generator=gen).to(kind).cuda()
    w = (t.randn((v, d), generator=gen) / d ** 0.5).to(kind).cuda()
    target = t.randint(0, v, (n,), generator=gen)
    target[1::4] = -100
    target, dloss = target.cuda(), t.randn(n, generator=gen).cuda()
    say(f"linear_ce {n}x{v}x{d} {dtype}")
    sizes = [og.linear_cross_entropy_workspace(n, v, d, CODES[dtype], grad) for grad in (False, True)]
    want = None
    for byte in (0, 0xFF, 0x7B):
        f, g = held(sizes[0], byte), held(sizes[1], byte)
        loss, lse = og.linear_cross_entropy(x, w, target, workspace=f[1])
        dx, dw = og.linear_cross_entropy_grad(x, w, target, lse, dloss, workspace=g[1])
        got = (loss, lse, dx, dw)
        assert all(r.isfinite().all() for r in got)
        assert untouched(f[0], sizes[0], byte) and untouched(g[0], sizes[1], byte)
        want = want or got
        assert all(t.equal(a, b) for a, b in zip(got, want)), byte


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("batch,m,n", [(1, 1, 1), (1, 33, 70), (3, 70, 33), (1, 300, 257), (2, 129, 400)])
def test_newton_schulz(batch, m, n, dtype):
    t = torch()
    g = t.randn((batch, m, n), generator=t.Generator().manual_seed(m)).to(getattr(t, dtype)).cuda()
    say(f"newton_schulz {batch} of {m}x{n} {dtype}")
    size = og.newton_schulz_workspace(batch, m, n, CODES[dtype])
    want = None
    for byte in (0, 0xFF, 0x7B):
        whole, ws = held(size, byte)
        got = og.newton_schulz(g, workspace=ws)
        assert got.isfinite().all() and untouched(whole, size, byte)
        want = got if want is None else want
        assert t.equal(got, want), byte
