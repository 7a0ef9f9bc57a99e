"""The Newton-Schulz update of matrices whose norm is far below eps: X starts at
nu = |G| / (|G| + eps) and keeps its bits there.

With X = nu Y the chain is that of Y from norm one with the coefficients
(a, b nu^2, c nu^4), whose result and bound lm_reference has; nu times both are
X's.  X's power of two is that of the next power of two above nu, up to 2 nu, so
that what a last bit costs is at most twice the reference's."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
A, B, C = 3.4445, -4.7750, 2.0315


def make(m, n, norm, dtype, seed):
    t = torch()
    g = t.randn((m, n), generator=t.Generator().manual_seed(seed), dtype=t.float64)
    return (g * (norm / g.norm())).to(getattr(t, dtype)).cuda()


def check(out, g, steps, eps, what):
    eps = float(torch().tensor(eps))  # as the call takes it, in fp32
    nu = float(g.double().norm() / (g.double().norm() + eps))
    exact, bound = ref.newton_schulz(g, steps, (A, B * nu ** 2, C * nu ** 4), 0.0)
    off = (out.double() - nu * exact).norm()
    assert off <= 2 * nu * bound, (f"{what}: off by {float(off / (nu * exact).norm()):.3g} of the result's norm, "
                                   f"bound {float(2 * bound / exact.norm()):.3g}")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("norm", [1e-7, 1e-10, 1e-12, 1e-14, 1e-16, 1e-23])
def test_norm_far_below_eps(norm, dtype):
    for m, n in ((1, 7), (40, 70), (130, 64), (300, 257)):
        say(f"newton_schulz {m}x{n} {dtype} |G| {norm}")
        g = make(m, n, norm, dtype, m + n)
        check(og.newton_schulz(g), g, 5, 1e-7, (m, n))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_many_steps_from_a_small_start(dtype):
    """The singular values grow by a per step until the polynomial holds them."""
    for m, n in ((40, 70), (300, 257)):
        say(f"newton_schulz {m}x{n} {dtype}")
        g = make(m, n, 1e-16, dtype, 1)
        for steps in (12, 20):
            check(og.newton_schulz(g, steps=steps), g, steps, 1e-7, (m, n, steps))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_norms_of_a_batch(dtype):
    """Each matrix of a batch has powers of its own: the bits of the call with that matrix alone."""
    t = torch()
    for m, n in ((40, 70), (300, 257)):
        say(f"newton_schulz {m}x{n} {dtype}")
        g = t.stack([make(m, n, norm, dtype, i) for i, norm in enumerate((1.0, 1e-14, 3.0, 1e-8, 1e-20))])
        g[2] = 0
        out = og.newton_schulz(g)
        assert (out[2] == 0).all()
        for i in (0, 1, 3, 4):
            check(out[i], g[i], 5, 1e-7, (m, n, i))
            assert t.equal(out[i], og.newton_schulz(g[i])), i


def test_a_large_eps():
    g = make(50, 90, 1.0, "float32", 3)
    for eps in (1.0, 1e3, 1e12):
        check(og.newton_schulz(g, eps=eps), g, 5, eps, eps)
