"""The 16-bit gradient of og_gemm_nt_epi with infinities and NaN in W, A and dC: every sum that they enter is
what the formula gives, on both sides of 128 rows."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu


def same_kinds(got, want):
    th = torch()
    got, inf = got.double(), float("inf")
    assert th.equal(got.isnan(), want.isnan())
    for side in (inf, -inf):
        assert th.equal(got == side, want == side)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
# (33, 2048, 64): dA in parts; (128, 40, 64) and above: more than one block of rows
@pytest.mark.parametrize("m,n,k", [(1, 40, 24), (16, 96, 64), (33, 2048, 64), (128, 40, 64), (129, 96, 64), (300, 17, 31)])
def test_infinities(m, n, k, act, dtype):
    th = torch()
    kind = getattr(th, dtype)
    gen = th.Generator().manual_seed(m + n)
    rnd = lambda *s: th.randn(s, generator=gen).to(kind).cuda()  # noqa: E731
    inf, nan = float("inf"), float("nan")
    dc, a, w, pre = rnd(m, n), rnd(m, k), rnd(n, k), rnd(m, n)
    pre = th.where(pre.abs() < 2 ** -5, th.full_like(pre, 0.5), pre)
    # a dP that the type holds: nothing remains of it
    dc[0], pre[0] = 1.0, 100.0
    w[3, 5], w[4, 6], w[7, 6], w[9, 8] = inf, -inf, inf, nan
    a[0, 3], a[m - 1, 4], a[m // 2, 7] = -inf, inf, nan
    say(f"gemm_nt_epi_grad infinities {m}x{n}x{k} {act} {dtype}")
    da, dw, db = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act=act)
    # (products term by term: an infinity times a slope of 0 is NaN)
    dp = dc.double() * ref.activation(pre.double(), act)[1]
    dp = th.where(dp.to(kind) == 0, th.zeros_like(dp), dp)
    want_a = th.stack([(row[:, None] * w.double()).sum(0) for row in dp])
    want_w = th.stack([(dp[:, j, None] * a.double()).sum(0) for j in range(n)])
    same_kinds(da, want_a)
    same_kinds(dw, want_w)
    assert db.isfinite().all()
    # dC's own
    w[3, 5] = w[4, 6] = w[7, 6] = w[9, 8] = 1
    a[0, 3] = a[m - 1, 4] = a[m // 2, 7] = 1
    dc[m // 2, 2], dc[m // 3, 11] = inf, nan
    pre[m // 2, 2] = 1.0
    da, dw, db = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act=act)
    dp = dc.double() * ref.activation(pre.double(), act)[1]
    same_kinds(da, th.stack([(row[:, None] * w.double()).sum(0) for row in dp]))
    same_kinds(dw, th.stack([(dp[:, j, None] * a.double()).sum(0) for j in range(n)]))
    same_kinds(db, dp.sum(0))
