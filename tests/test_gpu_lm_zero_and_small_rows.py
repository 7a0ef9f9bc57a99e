"""The fp32 cross entropy gradient where rows of X, W or dloss are zero or far
smaller than others, against 64 bits, each row of a gradient to its own size."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
IGNORE = -100


def make(n, v, d, seed, ignored=0.1):
    """Weights of 0.02, one weight 1/n for all rows, a target for each row."""
    t = torch()
    gen = t.Generator().manual_seed(seed)
    x = t.randn((n, d), generator=gen).cuda()
    w = (0.02 * t.randn((v, d), generator=gen)).cuda()
    target = t.randint(0, v, (n,), generator=gen)
    if n > 1:
        target[t.rand(n, generator=gen) < ignored] = IGNORE
    return x, w, target.cuda(), t.full((n,), 1.0 / n, device="cuda")


def bounds(x, w, target, dloss):
    """Exact dx and dw, and bounds of the call's errors.  With u = 2^-38 for half a last bit of a
    second plane against the largest value of what shares its power of two (2^13 units at least):

    - logits: the product's own errors, u of X's row for each weight, u of W's largest value for
      each value of X;
    - g: exp's argument and result as in lm_reference, 2^-22 in its planes, 2 u dloss_i (a row's
      largest g is 2^13 units at least, the powers of two to either side one more bit);
    - dx_i: g's errors and the sum's against W's absolute values, and |g_ij| u of W's largest;
    - dw_j: the same against X's rows, and |g_ij| 4 u of the largest |dloss| max |X| over
      dloss_i (two powers of two, each up to twice what it stands for)."""
    t, f = torch(), ref.F64
    keep = (target != IGNORE).nonzero()[:, 0]
    rows, w64, tk = x[keep].to(f), w.to(f), target[keep]
    dl = dloss[keep].to(f)[:, None]
    at = t.arange(len(keep), device=x.device)
    n, (v, d) = len(keep), w.shape
    u = ref.LAST
    z = rows @ w64.t()
    top_x, top_w = rows.abs().amax(1, keepdim=True), w64.abs().amax()
    ez = (rows.abs() @ w64.abs().t()) * ref.sum_error(d, 2)
    ez = ez + u * (top_x * w64.abs().sum(1) + rows.abs().sum(1, keepdim=True) * top_w)
    lse = t.logsumexp(z, 1)
    e = ref.cross_entropy(x, w, target, IGNORE, None)
    e_lse = e["e_lse"][keep][:, None]
    p = t.exp(z - lse[:, None])
    one = t.zeros_like(p)
    one[at, tk] = 1
    g = (p - one) * dl
    rel = t.expm1(ez + e_lse + (z - lse[:, None]).abs() * 2.0 ** -22 + 2.0 ** -22)
    eg = (p * rel + (p + one) * 2.0 ** -23) * dl.abs()
    eg = eg + (g.abs() + eg) * 2.0 ** -22 + 2 * u * dl.abs()
    ga = g.abs() + eg
    dx, e_dx = t.zeros(x.shape, dtype=f, device=x.device), t.zeros(x.shape, dtype=f, device=x.device)
    dx[keep] = g @ w64
    e_dx[keep] = eg @ w64.abs() + ga @ w64.abs() * (ref.sum_error(v, 2) + (16 + v / 2048) * ref.ADD) + \
        ga.sum(1, keepdim=True) * u * top_w
    dw = g.t() @ rows
    share = (dl.abs() * top_x).amax() / dl.abs().clamp(min=1e-300)
    e_dw = eg.t() @ rows.abs() + ga.t() @ rows.abs() * (ref.sum_error(n, 2) + 16 * ref.ADD) + \
        (ga.t() @ share.where(dl != 0, 0.0)) * 4 * u
    step, tiny = ref.half_step(t.float32), t.finfo(t.float32).tiny
    return (dx, e_dx + step * (dx.abs() + e_dx) + tiny), (dw, e_dw + step * (dw.abs() + e_dw) + tiny)


def check(x, w, target, dloss, what):
    loss, lse = og.linear_cross_entropy(x, w, target)
    e = ref.cross_entropy(x, w, target, IGNORE, None)
    assert ((lse.double() - e["lse"]).abs() <= e["e_lse"]).all(), what
    for got, name, (exact, bound) in zip(og.linear_cross_entropy_grad(x, w, target, lse, dloss),
                                         ("dx", "dw"), bounds(x, w, target, dloss)):
        off = (got.double() - exact).abs()
        bad = ~(off <= bound)
        assert not bad.any(), (f"{what} {name}: {int(bad.sum())} of {off.numel()} values off by up to "
                               f"{float((off / bound)[bad].max()):.3g} times the bound")


SIZES = [(1, 3, 5), (3, 17, 260), (5, 129, 64), (64, 512, 96), (300, 1024, 384), (700, 8191, 72)]


@pytest.mark.parametrize("n,v,d", SIZES + [(5000, 9001, 40)])
def test_ordinary_rows(n, v, d):
    say(f"linear_ce {n}x{v}x{d}")
    check(*make(n, v, d, 1), "ordinary")


@pytest.mark.parametrize("n,v,d", SIZES)
def test_zero_weights(n, v, d):
    """A head initialised with zeros: every probability is 1/v, dX is zero and dW is not."""
    say(f"linear_ce {n}x{v}x{d}")
    x, w, target, dloss = make(n, v, d, 2)
    check(x, w.zero_(), target, dloss, "W zero")


@pytest.mark.parametrize("n,v,d", SIZES)
def test_zero_activations(n, v, d):
    say(f"linear_ce {n}x{v}x{d}")
    x, w, target, dloss = make(n, v, d, 3)
    check(x.zero_(), w, target, dloss, "X zero")
    check(x, w.zero_(), target, dloss, "both zero")


@pytest.mark.parametrize("n,v,d", SIZES)
def test_zero_rows_among_others(n, v, d):
    """One counting row of X, padded rows of W, a row of W that is a target."""
    say(f"linear_ce {n}x{v}x{d}")
    for seed in (4, 5):
        x, w, target, dloss = make(n, v, d, seed, ignored=0.0)
        x[n // 2] = 0
        check(x, w, target, dloss, "a row of X")
        w[-min(12, v - 1):] = 0
        check(x, w, target, dloss, "and padded rows of W")
        w[target[0]] = 0
        check(x, w, target, dloss, "and a target's row of W")


@pytest.mark.parametrize("by", [-10, -20, -30, -60, 20])
def test_small_and_large_rows_to_their_own_size(by):
    """A few rows times 2^by: of W, of X and of dloss.  What a gradient's row is off by is
    bounded by its own terms; by other rows' only through 2^-38 of the largest value."""
    up = 2.0 ** by
    for n, v, d in ((5, 129, 64), (300, 1024, 384), (5000, 9001, 40)):
        say(f"linear_ce {n}x{v}x{d} times 2^{by}")
        x, w, target, dloss = make(n, v, d, 6)
        small = w.clone()
        small[::7] *= up
        check(x, small, target, dloss, "W")
        rows = x.clone()
        rows[::3] *= up
        if by < 0:
            check(rows, w, target, dloss, "X")
        weights = dloss.clone()
        weights[1::2] *= up
        weights[2::4] = 0
        check(x, w, target, weights, "dloss")
        if by < 0:
            check(rows, small, target, weights, "all")


def test_relative_error_of_small_rows():
    """Rows of W times 2^-20 and 2^-30 and, apart from them, rows of X and of dloss times 2^-20:
    their rows of the gradient keep the relative error that the others have.  Every term of these
    sums is off by at most 2^-17 of itself (probabilities of 2^-11 to 2^-9 keep 2^-22 of themselves,
    their logits of size 4 are off by less than 2^-18), and the sums' own size is their terms'
    over sqrt(n) or so: 2^-10 of the row's norm is far above, and far below what lost bits cost."""
    t = torch()
    x, w, target, dloss = make(256, 1024, 384, 7, ignored=0.0)
    for what, at, by in (("W", 3, 2.0 ** -20), ("W", 5, 2.0 ** -30), ("X", 7, 2.0 ** -20), ("dloss", 9, 2.0 ** -20)):
        a, b, dl = x.clone(), w.clone(), dloss.clone()
        {"W": b, "X": a, "dloss": dl}[what][at] *= by
        loss, lse = og.linear_cross_entropy(a, b, target)
        dx, dw = og.linear_cross_entropy_grad(a, b, target, lse, dl)
        (ex, _), (ew, _) = bounds(a, b, target, dl)
        got, want = (dw[at], ew[at]) if what == "W" else (dx[at], ex[at])
        assert (got.double() - want).norm() <= 2.0 ** -10 * want.norm(), (what, by)
