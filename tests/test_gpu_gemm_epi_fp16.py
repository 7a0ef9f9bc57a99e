"""The gradient of og_gemm_nt_epi in fp16 over its range: small dC, whose dP would be subnormal, dC near
the largest value, rows and columns of very different sizes, on both sides of 128 rows, against 64
bits."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
SMOOTH = ("gelu", "gelu_tanh", "silu")


def gradient(dc, a, w, pre, act):
    """Exact dA and dW and their bounds.  dP is held by a power of two of its row (for dA) or
    column (for dW) that brings the largest to 2^13 to 2^14: 2^-11 of each value, half of the
    last subnormal place 2^-25 at the least, 2^-38 of the largest.  Up to 128 rows the remainder, which
    is 2^-11 of the value or half of a subnormal place, is held to 2^-11 and 2^-25 again."""
    x, dc, a64, w64 = pre.to(ref.F64), dc.to(ref.F64), a.to(ref.F64), w.to(ref.F64)
    _, d = ref.activation(x, act)
    _, ed = ref.act_error(x, torch().zeros_like(x), act)
    dp = dc * d
    edp = dc.abs() * ed + 2.0 ** -24 * (dp.abs() + dc.abs() * ed) + 2.0 ** -149
    step = 2.0 ** -22 if len(dc) <= 128 else 2.0 ** -11
    out = []
    for p, e, right in ((dp, edp, w64.t()), (dp.t(), edp.t(), a64.t())):
        top = (p.abs() + e).amax(1, keepdim=True)
        held = e + step * (p.abs() + e) + 2.0 ** -38 * top
        exact = p @ right.t()
        bound = held @ right.abs().t() + ref.product_error(p, right, torch().float16) * 1.01
        out.append((exact, ref.rounded(exact, bound, torch().float16)))
    return out


def check(dc, a, w, pre, act):
    da, dw, _ = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act=act)
    for name, got, (want, bound) in zip(("da", "dw"), (da, dw), gradient(dc, a, w, pre, act)):
        off = (got.double() - want).abs()
        assert (off <= bound).all(), (name, (off / bound).max().item())
    return da, dw


def make(m, n, k, seed=0):
    th = torch()
    gen = th.Generator().manual_seed(seed + m + 3 * n + 7 * k)
    rnd = lambda *s: th.randn(s, generator=gen).cuda()  # noqa: E731
    return rnd(m, n), rnd(m, k), rnd(n, k), rnd(m, n).half()


# the last two: a product whose k is split, for dA and for dW
SIZES = [(5, 16, 24), (70, 24, 64), (128, 17, 33), (129, 16, 64), (300, 40, 72), (2100, 24, 40), (130, 4096, 64),
         (4096, 64, 64)]


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_small_gradients(m, n, k, act):
    """dC of 1e-6 is a few of fp16's last places; W and A are large, so that dA and dW are not."""
    dc, a, w, pre = make(m, n, k)
    for size in (1e-4, 1e-6):
        say(f"gemm_nt_epi_grad fp16 {m}x{n}x{k} {act} {size}")
        check((size * dc).half(), (100 * a).half(), (100 * w).half(), pre, act)


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_large_gradients(m, n, k, act):
    """dC near the largest fp16 times slopes above 1."""
    th = torch()
    dc, a, w, pre = make(m, n, k)
    dc = (65000 * dc.sign()).half()
    pre = th.where(pre > 0, th.full_like(pre, 1.5), pre)
    say(f"gemm_nt_epi_grad fp16 large {m}x{n}x{k} {act}")
    da, dw = check(dc, (1e-4 * a).half(), (1e-4 * w).half(), pre, act)
    assert da.isfinite().all() and dw.isfinite().all()


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("m,n,k", [(70, 60, 64), (300, 200, 64), (2100, 300, 40)])
def test_rows_and_columns_of_all_sizes(m, n, k, act):
    """dA's rows and dW's columns keep the bits of their own size."""
    th = torch()
    dc, a, w, pre = make(m, n, k)
    powers = lambda c: (2.0 ** th.linspace(-20, 13, c).round()).cuda()  # noqa: E731
    rows = powers(m)[:, None]
    say(f"gemm_nt_epi_grad fp16 rows {m}x{n}x{k} {act}")
    da, _ = check((dc * rows).half(), (1e-3 * a).half(), (0.05 * w).half(), pre, act)
    columns = powers(n)[None]
    say(f"gemm_nt_epi_grad fp16 columns {m}x{n}x{k} {act}")
    check((dc * columns).half(), (0.02 * a).half(), (1e-3 * w).half(), pre, act)


@pytest.mark.parametrize("m", [3, 70, 200])
def test_zero_and_special_rows(m):
    """Rows and columns of zeros stay zero; an infinity or NaN enters its row and column only."""
    th = torch()
    dc, a, w, pre = make(m, 48, 64)
    dc, a, w = dc.half(), a.half(), w.half()
    dc[0], dc[:, 5] = 0, 0
    for bad in (float("inf"), float("-inf"), float("nan")):
        dc[1, 7] = bad
        da, dw, db = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act="silu")
        assert (da[0] == 0).all() and (dw[5] == 0).all() and db[5] == 0
        assert not da[1].isfinite().any() and not dw[7].isfinite().any() and not db[7].isfinite()
        da[1], dw[7], db[7] = 0, 0, 0
        assert da.isfinite().all() and dw.isfinite().all() and db.isfinite().all()


def test_nothing_is_small_enough_to_be_lost():
    """A dC of the type's smallest value alone in its row."""
    th = torch()
    for m in (20, 200):
        dc = th.zeros((m, 40), device="cuda").half()
        dc[:, 3] = 2.0 ** -24
        pre = th.full_like(dc, -1.0)
        w, a = th.full((40, 64), 6e4, device="cuda").half(), th.full((m, 64), 6e4, device="cuda").half()
        check(dc, a, w, pre, "silu")
