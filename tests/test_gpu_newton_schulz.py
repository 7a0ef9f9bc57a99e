"""The Newton-Schulz update against 64 bits."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
COEFFS = (3.4445, -4.7750, 2.0315)


def make(shape, dtype, seed=0, scale=0.01):
    t = torch()
    gen = t.Generator().manual_seed(seed)
    rank = max(1, min(shape[-2:]) // 4)
    g = t.randn((*shape[:-1], rank), generator=gen) @ t.randn((*shape[:-2], rank, shape[-1]), generator=gen)
    g = g / rank ** 0.5 + 0.3 * t.randn(shape, generator=gen)
    return (scale * g).to(getattr(t, dtype)).cuda()


def check(out, g, steps=5, coeffs=COEFFS, eps=1e-7, what=""):
    m, n = g.shape[-2:]
    for o, one in zip(out.reshape(-1, m, n), g.reshape(-1, m, n)):
        exact, bound = ref.newton_schulz(one, steps, coeffs, eps)
        off = (o.double() - exact).norm()
        assert off <= bound, f"{what}: off by {float(off):.3g}, bound {float(bound):.3g}"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (7, 1), (5, 5), (64, 64), (65, 64), (63, 200), (200, 63),
                                 (129, 130), (130, 300), (300, 257), (513, 520), (33, 1000)])
def test_shapes(m, n, dtype):
    say(f"newton_schulz {m}x{n} {dtype}")
    g = make((m, n), dtype, seed=m + n)
    check(og.newton_schulz(g), g, what=(m, n, dtype))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("steps", [1, 2, 3])
def test_few_steps_and_other_coefficients(steps, dtype):
    """One step is tight enough to show a wrong polynomial; the cubic has c = 0."""
    for coeffs in (COEFFS, (1.5, -0.5, 0.0), (1.0, 0.0, 0.0), (2.0, -1.5, 0.5)):
        g = make((90, 150), dtype, seed=steps)
        check(og.newton_schulz(g, steps=steps, coeffs=coeffs), g, steps, coeffs, what=(steps, coeffs))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_large_tiles(dtype):
    for shape in ((1100, 1300), (2304, 768)):
        say(f"newton_schulz {shape} {dtype}")
        g = make(shape, dtype, seed=3)
        check(og.newton_schulz(g), g, what=shape)


@pytest.mark.parametrize("dtype,r,k,batch", [
    ("bfloat16", 257, 257, 1), ("bfloat16", 331, 331, 32), ("bfloat16", 405, 405, 48),
    ("bfloat16", 331, 531, 64), ("bfloat16", 257, 514, 12), ("bfloat16", 479, 479, 64),
    ("float32", 130, 130, 24), ("float32", 200, 200, 64), ("float32", 331, 331, 64),
    ("float32", 405, 405, 48), ("float32", 997, 997, 16), ("bfloat16", 200, 200, 64),
])
def test_every_tile(dtype, r, k, batch):
    """Batches that together bring each product to each of its tiles: two matrices in turn, all of
    whose results repeat bit for bit."""
    t = torch()
    say(f"newton_schulz {batch} of {r}x{k} {dtype}")
    two = make((2, r, k), dtype, seed=r + k)
    out = og.newton_schulz(two[t.arange(batch) % 2], steps=2)
    check(out[:2], two[:batch], steps=2, what=(r, k, batch))
    for b in range(2, batch):
        assert t.equal(out[b], out[b % 2]), b


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_batches_views_and_gaps(dtype):
    t = torch()
    g = make((2, 3, 40, 70), dtype, seed=4)
    out = og.newton_schulz(g)
    check(out, g, what="batch")
    for b in range(3):
        assert t.equal(og.newton_schulz(g[1, b]), out[1, b])
    big = t.full((6, 43, 79), float("nan"), dtype=g.dtype, device="cuda")
    view = big[:, 2:42, 5:75]
    view.copy_(g.view(6, 40, 70))
    dst = t.full((6, 44, 75), 7.5, dtype=g.dtype, device="cuda")
    og.newton_schulz(view, out=dst[:, 1:41, 3:73])
    assert t.equal(dst[:, 1:41, 3:73], out.view(6, 40, 70))
    mask = t.ones_like(dst, dtype=t.bool)
    mask[:, 1:41, 3:73] = False
    assert (dst[mask] == 7.5).all()
    # one input for the whole batch
    same = og.newton_schulz(g[0, 0].expand(3, 40, 70), out=t.empty((3, 40, 70), dtype=g.dtype, device="cuda"))
    assert all(t.equal(s, out[0, 0]) for s in same)
    # in place
    own = g.clone()
    assert og.newton_schulz(own, out=own) is own
    assert t.equal(own, out)


def test_empty_zero_and_not_finite():
    t = torch()
    assert og.newton_schulz(t.empty((0, 5), device="cuda")).shape == (0, 5)
    assert og.newton_schulz(t.empty((4, 0), device="cuda")).shape == (4, 0)
    assert og.newton_schulz(t.empty((0, 4, 5), device="cuda")).shape == (0, 4, 5)
    for dtype in (t.float32, t.bfloat16):
        assert (og.newton_schulz(t.zeros((30, 40), dtype=dtype, device="cuda")) == 0).all()
        g = make((2, 30, 40), str(dtype)[6:], seed=5)
        g[1, 3, 4] = float("nan")
        out = og.newton_schulz(g)
        assert out[0].isfinite().all() and out[1].isnan().all()
        g[1, 3, 4] = float("inf")
        assert og.newton_schulz(g)[1].isnan().all()


@pytest.mark.parametrize("scale", [1e-30, 1e18])
def test_small_and_large_values(scale):
    """The norm's squares leave fp32's range; 1e-30 with the eps of an exact zero."""
    g = make((50, 60), "float32", seed=6, scale=scale)
    check(og.newton_schulz(g, eps=0.0), g, eps=0.0, what=scale)


def test_orthogonal_in_the_limit():
    """The classical cubic step brings every singular value to one: X X^T - I after 30 steps is
    what fp32 products leave (derived: sum_error of a product of r x r values of size one)."""
    t = torch()
    gen = t.Generator().manual_seed(7)
    g = t.randn((48, 200), generator=gen).cuda()
    x = og.newton_schulz(g, steps=30, coeffs=(1.5, -0.5, 0.0)).double()
    off = (x @ x.t() - t.eye(48, device="cuda", dtype=t.float64)).norm()
    # the last step's own errors, and half of the error before it is kept (p'(1) = 0 for the
    # stretch, 1 for a rotation, which leaves X X^T as it is)
    a = x.abs()
    local = ref.sum_error(200, 2) * (a @ a.t()).norm() * 0.5 + ref.sum_error(48, 2) * a.norm() * 48 ** 0.5 + \
        (2.0 ** -22 + 4 * 2.0 ** -24) * a.norm() + (2.0 ** -22 + ref.LAST * 48) * 48 ** 0.5
    assert off <= 2 * 2 * local


def test_same_bits_every_run():
    t = torch()
    g = make((300, 700), "bfloat16", seed=8)
    first = og.newton_schulz(g)
    for _ in range(3):
        assert t.equal(og.newton_schulz(g), first)
