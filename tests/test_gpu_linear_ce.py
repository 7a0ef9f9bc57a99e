"""The linear cross entropy and its gradient against 64 bits."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
IGNORE = -100


def make(n, v, d, dtype, ignored=0.2, seed=0, scale=2.0):
    t = torch()
    gen = t.Generator().manual_seed(seed)
    kind = getattr(t, dtype)
    x = t.randn((n, d), generator=gen).to(kind).cuda()
    w = (t.randn((v, d), generator=gen) * scale / d ** 0.5).to(kind).cuda()
    target = t.randint(0, v, (n,), generator=gen)
    target[t.rand(n, generator=gen) < ignored] = IGNORE
    dloss = t.randn(n, generator=gen).cuda()
    return x, w, target.cuda(), dloss


def within(got, exact, bound, what):
    off = (got.double() - exact).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {off.numel()} values off by up to "
                           f"{float((off / bound)[bad].max()):.3g} times the bound")


def check(x, w, target, dloss, ignore=IGNORE, got=None):
    loss, lse = og.linear_cross_entropy(x, w, target, ignore_index=ignore)
    dx, dw = og.linear_cross_entropy_grad(x, w, target, lse, dloss, ignore_index=ignore)
    e = ref.cross_entropy(x, w, target, ignore, dloss)
    within(loss, e["loss"], e["e_loss"], "loss")
    within(lse, e["lse"], e["e_lse"], "lse")
    within(dx, e["dx"], e["e_dx"], "dx")
    within(dw, e["dw"], e["e_dw"], "dw")
    return loss, lse, dx, dw


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,v,d", [
    (1, 1, 1), (1, 2, 3), (2, 257, 7), (3, 1000, 64), (5, 63, 65), (64, 64, 64), (65, 129, 72),
    (130, 300, 200), (257, 2049, 8), (300, 513, 1000), (700, 4099, 130), (1, 5000, 256),
    (1100, 100, 33), (17, 33000, 24), (40, 3000, 4100),
])
def test_shapes(n, v, d, dtype):
    say(f"linear_ce {n}x{v}x{d} {dtype}")
    check(*make(n, v, d, dtype, seed=n + v + d))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_several_pieces_of_the_vocabulary(dtype):
    """More columns than a piece holds, the last piece ragged."""
    n, v, d = 5000, 9001, 40
    say(f"linear_ce {n}x{v}x{d} {dtype}")
    check(*make(n, v, d, dtype, seed=1))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,v,d", [(9000, 9001, 24), (9000, 9001, 25), (20000, 9001, 72), (40, 9001, 8200)])
def test_two_and_three_pieces(n, v, d, dtype):
    """dX summed over two and three pieces (a piece holds 2^26 values of g or of W), with its sum
    over a piece whole or (the last) split; d = 25: bf16 weights that are copied first."""
    say(f"linear_ce {n}x{v}x{d} {dtype}")
    check(*make(n, v, d, dtype, seed=n + d))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9])
def test_few_rows(n, dtype):
    """Rows around those that a kernel of their own takes, layers that give each wave many rows
    and none, columns that end inside a load, rows that do not count among them and strides that
    are not whole loads."""
    t = torch()
    for v, d in ((1, 3), (17, 260), (1023, 255), (1025, 64), (5003, 1000), (40000, 65)):
        x, w, target, dloss = make(n, v, d, dtype, seed=n + v, ignored=0.3)
        say(f"linear_ce {n}x{v}x{d} {dtype}")
        loss, lse, dx, dw = check(x, w, target, dloss)
        for need in ((True, False), (False, True)):
            one = og.linear_cross_entropy_grad(x, w, target, lse, dloss, need=need)
            assert all(a is None or t.equal(a, b) for a, b in zip(one, (dx, dw)))
        wide = t.full((v, d + 3), float("nan"), dtype=w.dtype, device="cuda")[:, 1:d + 1]
        wide.copy_(w)
        check(x, wide, target, dloss)
        target.fill_(IGNORE)
        loss, lse, dx, dw = check(x.fill_(float("nan")), w, target, dloss)
        assert (dx == 0).all() and (dw == 0).all() and (loss == 0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n,v,d", [
    (4000, 5000, 776), (1000, 5000, 4104), (9000, 100, 776), (9000, 100, 1000), (500, 1300, 4104),
    (20000, 900, 264), (5000, 100, 2056),
])
def test_every_tile(n, v, d, dtype):
    """Sizes that together bring each product of the operator to each of its tiles."""
    say(f"linear_ce {n}x{v}x{d} {dtype}")
    check(*make(n, v, d, dtype, seed=n + v))


def test_rows_of_all_sizes():
    """fp32 rows of X and W and values of dloss from tiny to large and zero, each row of the
    planes to a power of its own."""
    t = torch()
    x, w, target, dloss = make(140, 260, 72, "float32", seed=13)
    gen = t.Generator().manual_seed(14)
    up = 2.0 ** t.randint(-60, 61, (140, 1), generator=gen).cuda()
    x, w = x * up / 2.0 ** 60, w * 2.0 ** t.randint(-100, 5, (260, 1), generator=gen).cuda()
    x[7], w[11], dloss[13] = 0, 0, 0
    dloss *= 2.0 ** t.randint(-30, 31, (140,), generator=gen).cuda()
    check(x, w, target, dloss)
    dloss.zero_()
    loss, lse, dx, dw = check(x, w, target, dloss)
    assert (dx == 0).all() and (dw == 0).all()
    x.zero_()
    check(x, w, target, dloss)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_large_tiles(dtype):
    n, v, d = 1500, 12000, 136
    say(f"linear_ce {n}x{v}x{d} {dtype}")
    check(*make(n, v, d, dtype, seed=2, ignored=0.5))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_ignored_rows_hold_anything(dtype):
    """NaN and infinities in ignored rows of X, lse and dloss reach nothing; the others' results
    are the bits of the call without those rows."""
    t = torch()
    x, w, target, dloss = make(150, 400, 96, dtype, seed=3, ignored=0.4)
    drop = target == IGNORE
    clean = check(x, w, target, dloss)
    x2, dl2 = x.clone(), dloss.clone()
    x2[drop] = float("nan")
    x2[drop.nonzero()[0], ::2] = float("inf")
    dl2[drop] = float("nan")
    loss, lse = og.linear_cross_entropy(x2, w, target, ignore_index=IGNORE)
    lse2 = lse.clone()
    lse2[drop] = float("nan")
    dx, dw = og.linear_cross_entropy_grad(x2, w, target, lse2, dl2, ignore_index=IGNORE)
    for a, b in zip((loss, lse, dx, dw), clean):
        assert t.equal(a, b)
    assert (loss[drop] == 0).all() and (lse[drop] == 0).all() and (dx[drop] == 0).all()
    keep = ~drop
    loss3, lse3 = og.linear_cross_entropy(x[keep].contiguous(), w, target[keep].contiguous())
    assert t.equal(loss3, loss[keep]) and t.equal(lse3, lse[keep])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_all_rows_ignored_and_none(dtype):
    t = torch()
    x, w, target, dloss = make(70, 90, 48, dtype, seed=4)
    target.fill_(IGNORE)
    loss, lse, dx, dw = check(x, w, target, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    empty = (x[:0], w, target[:0])
    loss, lse = og.linear_cross_entropy(*empty)
    assert loss.shape == (0,)
    dw = t.full_like(w, 3)
    dx, got = og.linear_cross_entropy_grad(*empty, lse, dloss[:0], dW=dw)
    assert got is dw and (dw == 0).all() and dx.shape == (0, 48)


def test_targets_outside_the_vocabulary_and_an_ignore_index_inside():
    t = torch()
    x, w, target, dloss = make(60, 50, 32, "float32", seed=5, ignored=0)
    target[3], target[4], target[5] = 50, -7, 1 << 40
    loss, lse = og.linear_cross_entropy(x, w, target, ignore_index=7)
    dx, dw = og.linear_cross_entropy_grad(x, w, target, lse, dloss, ignore_index=7)
    e = ref.cross_entropy(x, w, target, 7, dloss)
    bad = t.zeros(60, dtype=t.bool, device="cuda")
    bad[3:6] = True
    assert loss[bad].isnan().all() and (lse[bad] == 0).all() and (dx[bad] == 0).all()
    within(loss[~bad], e["loss"][~bad], e["e_loss"][~bad], "loss")
    within(dx, e["dx"], e["e_dx"], "dx")
    within(dw, e["dw"], e["e_dw"], "dw")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_strides_offsets_and_gaps(dtype):
    """Odd row strides and offsets (no 16-byte alignment), NaN in the inputs' gaps, a sentinel in
    the outputs' that must survive."""
    t = torch()
    n, v, d = 75, 210, 56
    x, w, target, dloss = make(n, v, d, dtype, seed=6)
    for pad, at in ((8, 0), (8, 8), (5, 3), (1, 1)):
        bx = t.full((n, d + pad), float("nan"), dtype=x.dtype, device="cuda")
        bw = t.full((v, d + pad), float("nan"), dtype=x.dtype, device="cuda")
        bx[:, at:at + d], bw[:, at:at + d] = x, w
        gx = t.full((n, d + pad + 2), 7.5, dtype=x.dtype, device="cuda")
        gw = t.full((v, d + pad + 2), 7.5, dtype=x.dtype, device="cuda")
        vx, vw = bx[:, at:at + d], bw[:, at:at + d]
        loss, lse = og.linear_cross_entropy(vx, vw, target)
        og.linear_cross_entropy_grad(vx, vw, target, lse, dloss, dX=gx[:, 1:1 + d], dW=gw[:, 1:1 + d])
        e = ref.cross_entropy(x, w, target, IGNORE, dloss)
        within(loss, e["loss"], e["e_loss"], "loss")
        within(gx[:, 1:1 + d], e["dx"], e["e_dx"], "dx")
        within(gw[:, 1:1 + d], e["dw"], e["e_dw"], "dw")
        for b in (gx, gw):
            assert (b[:, :1] == 7.5).all() and (b[:, 1 + d:] == 7.5).all()


def test_one_gradient_alone():
    t = torch()
    x, w, target, dloss = make(90, 110, 40, "bfloat16", seed=7)
    loss, lse, dx, dw = check(x, w, target, dloss)
    only = og.linear_cross_entropy_grad(x, w, target, lse, dloss, need=(True, False))
    assert only[1] is None and t.equal(only[0], dx)
    only = og.linear_cross_entropy_grad(x, w, target, lse, dloss, need=(False, True))
    assert only[0] is None and t.equal(only[1], dw)


def test_large_logits():
    """Logits of some hundreds: exp of most of them underflows, none overflows."""
    x, w, target, dloss = make(80, 300, 64, "float32", seed=8, scale=200.0)
    check(x, w, target, dloss)


def test_a_value_that_is_not_finite_shows():
    t = torch()
    x, w, target, dloss = make(70, 100, 32, "bfloat16", seed=9, ignored=0)
    x[11, 3] = float("nan")
    loss, lse = og.linear_cross_entropy(x, w, target)
    assert loss[11].isnan() and int(loss.isnan().sum()) == 1


def test_gradient_against_differences():
    """dX and dW along random directions against central differences of the 64-bit loss.  The
    difference is off by h^2/6 of a third derivative: every logit's derivatives along the
    direction u are at most |u_z|^3 of order one, summed over the rows' weights."""
    t = torch()
    x, w, target, dloss = make(50, 70, 24, "float32", seed=10)
    loss, lse = og.linear_cross_entropy(x, w, target)
    dx, dw = og.linear_cross_entropy_grad(x, w, target, lse, dloss)
    e = ref.cross_entropy(x, w, target, IGNORE, dloss)
    keep = target != IGNORE

    def total(x64, w64):
        z = x64[keep] @ w64.t()
        return (dloss.double()[keep] * (t.logsumexp(z, 1) - z.gather(1, target[keep][:, None])[:, 0])).sum()

    gen = t.Generator(device="cuda").manual_seed(1)
    h = 1e-4
    for _ in range(4):
        u = t.randn(x.shape, generator=gen, device="cuda", dtype=t.float64)
        s = t.randn(w.shape, generator=gen, device="cuda", dtype=t.float64)
        for ux, uw in ((u, 0 * s), (0 * u, s)):
            x64, w64 = x.double(), w.double()
            diff = (total(x64 + h * ux, w64 + h * uw) - total(x64 - h * ux, w64 - h * uw)) / (2 * h)
            got = (dx.double() * ux).sum() + (dw.double() * uw).sum()
            zs = (ux[keep] @ w64.t() + x64[keep] @ uw.t()).abs().amax(1) * 2
            third = (dloss.double()[keep].abs() * zs ** 3).sum() * h * h
            bound = (e["e_dx"] * ux.abs()).sum() + (e["e_dw"] * uw.abs()).sum() + third + 1e-9
            assert (got - diff).abs() <= bound


def test_a_common_weight_costs_no_bits():
    """bf16: all rows with the weight c against all with 1.  Both are the same sums, c times and
    rounded to bf16 once each, half a step (and fp32's roundings) apart; c = 1 + 2^-8 is the
    number that a rounding to bf16 would move most."""
    t = torch()
    x, w, target, dloss = make(200, 500, 64, "bfloat16", seed=15)
    loss, lse = og.linear_cross_entropy(x, w, target)
    c = 1 + 2.0 ** -8
    one = og.linear_cross_entropy_grad(x, w, target, lse, t.ones_like(dloss))
    two = og.linear_cross_entropy_grad(x, w, target, lse, t.full_like(dloss, c))
    for a, b in zip(one, two):
        a, b = a.double(), b.double()
        within(b, c * a, ref.half_step(t.bfloat16) * (c * a.abs() + b.abs()) * (1 + 2.0 ** -20), "weight")


def test_same_bits_every_run():
    t = torch()
    x, w, target, dloss = make(400, 1500, 128, "bfloat16", seed=11)
    first = check(x, w, target, dloss)
    for _ in range(3):
        loss, lse = og.linear_cross_entropy(x, w, target)
        again = (loss, lse, *og.linear_cross_entropy_grad(x, w, target, lse, dloss))
        assert all(t.equal(a, b) for a, b in zip(first, again))


def test_rows_past_32_bits():
    """Rows of W further than 2^32 bytes apart in one tile, read in place and by planes."""
    t = torch()
    for dtype in ("bfloat16", "float32"):
        x, w, target, dloss = make(30, 80, 64, dtype, seed=12)
        stride = 1 << 22
        flat = t.empty(79 * stride + 64, dtype=w.dtype, device="cuda")
        far = t.as_strided(flat, w.shape, (stride, 1))
        far.copy_(w)
        loss, lse = og.linear_cross_entropy(x, far, target)
        dx, dw = og.linear_cross_entropy_grad(x, far, target, lse, dloss)
        e = ref.cross_entropy(x, w, target, IGNORE, dloss)
        within(loss, e["loss"], e["e_loss"], "loss")
        within(dx, e["dx"], e["e_dx"], "dx")
        within(dw, e["dw"], e["e_dw"], "dw")
        del flat, far
