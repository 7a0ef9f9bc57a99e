"""The gradient of og_gemm_nt_epi in bf16 with a smooth activation: dP's bits beyond bf16's are kept, on both
sides of 128 and 384 rows, for rows and columns of all sizes, against 64 bits."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
SMOOTH = ("gelu", "gelu_tanh", "silu")


def gradient(dc, a, w, pre, act):
    """Exact dA, dW and dbias for this pre, and bounds.  Up to 384 rows dP is held to 2^-8 of it and its remainder
    to 2^-8 of that, both down to bf16's smallest; of more rows in fp16 to 2^-11, and it and the other
    operand (whose 8 bits fp16 holds) down to half of the last subnormal place, 2^-25, where the largest of
    the row or column is 2^13 at the least."""
    th = torch()
    x, dc, a64, w64 = pre.to(ref.F64), dc.to(ref.F64), a.to(ref.F64), w.to(ref.F64)
    _, d = ref.activation(x, act)
    _, ed = ref.act_error(x, th.zeros_like(x), act)
    dp = dc * d
    edp = dc.abs() * ed + 2.0 ** -24 * (dp.abs() + dc.abs() * ed) + 2.0 ** -149
    few = len(dc) <= 384
    out = []
    for p, e, right in ((dp, edp, w64.t()), (dp.t(), edp.t(), a64.t())):
        size = p.abs() + e
        held = e + (2.0 ** -16 if few else 2.0 ** -11) * size + 2.0 ** -133
        lost = th.zeros_like(right[:, :1])
        if not few:
            held = held + 2.0 ** -38 * size.amax(1, keepdim=True)
            lost = 2.0 ** -38 * right.abs().amax(1, keepdim=True)
        exact = p @ right.t()
        bound = held @ right.abs().t() + (size + held) @ lost.expand_as(right).t()
        bound = bound + ref.product_error(p, right, th.bfloat16) * 1.02
        out.append((exact, ref.rounded(exact, bound, th.bfloat16)))
    db = dp.sum(0)
    return out + [(db, ref.rounded(db, edp.sum(0) + 22 * 2.0 ** -24 * (dp.abs() + edp).sum(0), th.bfloat16))]


def check(dc, a, w, pre, act):
    got = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act=act)
    for name, t, (want, bound) in zip(("da", "dw", "dbias"), got, gradient(dc, a, w, pre, act)):
        off = (t.double() - want).abs()
        assert (off <= bound).all(), (name, (off / bound).max().item())
    return got


def make(m, n, k, seed=0):
    th = torch()
    gen = th.Generator().manual_seed(seed + m + 3 * n + 7 * k)
    rnd = lambda *s: th.randn(s, generator=gen).bfloat16().cuda()  # noqa: E731
    return rnd(m, n), rnd(m, k), rnd(n, k), rnd(m, n)


# (130 and 400 by 4096: dA with k in parts; 4100: dW)
SIZES = [(5, 16, 24), (128, 17, 33), (129, 16, 64), (384, 24, 40), (385, 24, 40), (385, 17, 33), (500, 40, 72), (130, 4096, 64),
         (400, 4096, 64), (4100, 24, 40), (8300, 16, 16)]


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("size", [1.0, 1e-6, 1e-30])
def test_bits_of_dp(m, n, k, act, size):
    """Few columns of dA's sums and few rows of dW's are not 0, so that single roundings show."""
    dc, a, w, pre = make(m, n, k)
    if n > 1000:
        dc[:, 16:] = 0
    dc[1:] *= (torch().arange(1, m, device="cuda") % (m // 16 + 1) == 0)[:, None]
    say(f"gemm_nt_epi_grad bf16 {m}x{n}x{k} {act} {size}")
    check((dc * size).bfloat16(), a, w, pre, act)


@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("m,n,k", [(300, 200, 64), (700, 150, 64), (2100, 300, 40)])
def test_rows_and_columns_of_all_sizes(m, n, k, act):
    """dA's rows and columns and dW's rows and columns keep the bits of their own size."""
    th = torch()
    powers = lambda c: (2.0 ** th.linspace(-60, 50, c).round()).bfloat16().cuda()  # noqa: E731
    dc, a, w, pre = make(m, n, k)
    say(f"gemm_nt_epi_grad bf16 sizes {m}x{n}x{k} {act}")
    check(dc * powers(m)[:, None], (a * 1e-20).bfloat16(), w * powers(k)[None], pre, act)
    check(dc * powers(n)[None], a * powers(k)[None], (w * 1e-20).bfloat16(), pre, act)


@pytest.mark.parametrize("m", [200, 400, 8200])
def test_parts_zeros_and_special_values(m):
    """Each of the three alone is the same; rows and columns of zeros; infinities and NaN of dC, W and A enter what
    the formula says."""
    th = torch()
    dc, a, w, pre = make(m, 48, 64)
    dc[0], dc[:, 5] = 0, 0
    every = check(dc, a, w, pre, "silu")
    assert (every[0][0] == 0).all() and (every[1][5] == 0).all() and every[2][5] == 0
    for need in [(True, False, False), (False, True, False), (False, False, True), (True, True, False)]:
        got = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act="silu", need=need)
        assert all(g is None if not n else th.equal(g, e) for g, e, n in zip(got, every, need))
    inf, nan = float("inf"), float("nan")
    w[3, 9], w[4, 10], w[6, 11], a[7, 20], a[8, 21], a[9, 22] = inf, -inf, nan, inf, -inf, nan
    dc[20, 30], dc[21, 31] = inf, nan
    da, dw, db = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act="silu")
    dp = dc.double() * ref.activation(pre.double(), "silu")[1]
    want_a = sum(dp[:, j, None] * w[j].double() for j in range(48))
    want_w = th.stack([(dp[:, j, None] * a.double()).sum(0) for j in range(48)])
    for got, want in ((da, want_a), (dw, want_w), (db, dp.sum(0))):
        got = got.double()
        assert th.equal(got.isnan(), want.isnan()) and th.equal(got == inf, want == inf)
        assert th.equal(got == -inf, want == -inf)


@pytest.mark.parametrize("m,n,k", [(385, 33, 70), (600, 200, 128)])
def test_workspace_and_strides(m, n, k):
    """A workspace holds anything before; operands inside wider matrices at odd offsets give the same."""
    th = torch()
    dc, a, w, pre = make(m, n, k)
    want = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act="gelu")
    size = og.gemm_nt_epi_workspace(m, n, k, og.BF16, True)
    held = th.full((size + 8192,), 0x7B, dtype=th.uint8, device="cuda")
    got = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act="gelu", workspace=held[4096:4096 + size])
    assert all(th.equal(x, y) for x, y in zip(got, want))
    assert (held[:4096] == 0x7B).all() and (held[4096 + size:] == 0x7B).all()

    def wide(t):
        big = th.full((t.shape[0], t.shape[1] + 9), 1e3, dtype=t.dtype, device="cuda")
        big[:, 3:3 + t.shape[1]] = t
        return big[:, 3:3 + t.shape[1]]

    got = og.gemm_nt_epi_grad(wide(dc), wide(a), wide(w), pre=wide(pre), act="gelu")
    assert all(th.equal(x, y) for x, y in zip(got, want))
