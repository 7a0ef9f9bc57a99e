"""The activations of og_gemm_nt_epi and their slopes to a relative error in both tails, where the values are
far below their arguments, against 64 bits."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

SMOOTH = ("gelu", "gelu_tanh", "silu")
EVERY = ("float32", "bfloat16", "float16")
UNIT = 2.0 ** -23  # the exponential's and the reciprocal's error; an operation's rounding is half of it


def points(dtype):
    th = torch()
    ends = [c + d for c in (-130.0, -88.0, -87.0, -80.0, -20.0, -13.2, -10.0, -5.5, 0.0) for d in (-0.07, -0.01, 0.0, 0.01, 0.07)]
    x = th.cat([th.linspace(-130, 130, 5001), th.linspace(-21, 21, 6001), th.logspace(-30, 2, 500), -th.logspace(-30, 2, 500),
                th.tensor(ends), -th.tensor(ends)])
    return x.to(getattr(th, dtype)).unique()


def bounds(x, act, dtype):
    """act(x), act'(x) in 64 bits and their bounds.

    An exponential e^-t by 2^(-t log2 e) has the relative error of its argument's operations and
    constants (half a UNIT each) times t, and a UNIT: SiLU two of t = |x|, GELU three of
    x^2 / 2, GELU by tanh seven of t = |u|.  SiLU and tanh: a sum, a reciprocal and a product besides, 3 UNIT in all.
    GELU's tail besides: s 1.5, to which the tail moves 3 times as much at most; the polynomial 0.7, its
    steps 6, three products 1.5, e 1: 14.  The slopes are sums of two terms whose sizes the bound
    takes, each of at most twice these errors and a few operations.  Factors below 2^-126 are 0;
    the slope is 0 or 1 beyond 80 (SiLU), 20 and 10, where it is that to 2^-108, 2^-200 and 2^-116."""
    th = torch()
    x = x.double()
    kind = getattr(th, dtype)
    y, d = ref.activation(x, act)
    a = x.abs()
    if act == "silu":
        below, above = th.sigmoid(x), th.sigmoid(-x)
        times, size, flat = a + 4, below + a * below * above, 2.0 ** -108
    elif act == "gelu":
        below = 0.5 * th.erfc(-x * 0.5 ** 0.5)
        size = below + a * th.exp(-x * x / 2) * 0.4
        times, flat = 0.75 * x * x + 14, 0.0
    else:
        u = 2 * (2 / th.pi) ** 0.5 * (x + 0.044715 * x ** 3)
        below, above = th.sigmoid(u), th.sigmoid(-u)
        size = below + a * below * above * 1.6 * (1 + 3 * 0.044715 * x * x)
        times, flat = 3.5 * u.abs() + 4, 2.0 ** -116
    times = times.clamp(max=1e4)  # (beyond, values are 0 or x)
    lost = 2.0 ** -126 * (1 + a)
    e_y = times * UNIT * y.abs() + lost
    e_d = (2 * times + 8) * UNIT * size + lost * (1 + a + x * x).clamp(max=1e3) + flat
    return y, ref.rounded(y, e_y, kind), d, ref.rounded(d, e_d, kind)


@pytest.mark.parametrize("act", SMOOTH)
def test_bounds_see_a_lost_tail(act):
    """A tail that is 0 below -5.5 (SiLU: -17), and values to an absolute error of fp32's, are outside."""
    th = torch()
    x = points("float32").double()
    y, e_y, d, e_d = bounds(x, act, "float32")
    # (fp32 holds values down to 2^-126; far right the slope is 1, far left it passes through 0)
    tail = (x < (-17 if act == "silu" else -5.5)) & (y.abs() > 2.0 ** -100)
    assert tail.sum() > 50
    assert (y.abs() > 100 * e_y)[tail].all() and (d.abs() > 100 * e_d)[tail].all()
    near = (x < -6) & (x > -7) if act != "silu" else (x < -20) & (x > -21)
    assert near.any() and (2.0 ** -25 > 10 * e_y)[near].all() and (2.0 ** -25 > 10 * e_d)[near].all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", SMOOTH)
@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("m", [1, 100, 200])
def test_tails(act, dtype, m):
    """v is the bias alone where A is zero (m: the kernel of few rows, tiles); dbias of a dC with one row
    of ones is the slope."""
    th = torch()
    kind = getattr(th, dtype)
    x = points(dtype).cuda()
    n = len(x)
    A, B = th.zeros((m, 256), dtype=kind, device="cuda"), th.ones((n, 256), dtype=kind, device="cuda")
    say(f"gemm_nt_epi tails {dtype} {act} {m}")
    out, pre = og.gemm_nt_epi(A, B, bias=x, act=act, need_pre=True)
    assert all(th.equal(row, x) for row in pre[:: max(1, m // 3)])
    y, e_y, d, e_d = bounds(x, act, dtype)
    off = (out.double() - y).abs()
    assert (off <= e_y).all(), (x[(off / e_y).amax(0).argmax()].item(), (off / e_y).max().item())
    dc = th.zeros_like(out)
    dc[m // 2] = 1
    db = og.gemm_nt_epi_grad(dc, A, B, pre=pre, act=act, need=(False, False, True))[2]
    off = (db.double() - d).abs()
    assert (off <= e_d).all(), (x[(off / e_d).argmax()].item(), (off / e_d).max().item())
