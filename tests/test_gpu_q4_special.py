"""The product with 4-bit weights: infinite and NaN scales, activations at the
ends of their types and every zero point, through each of its kernels (by rows
of A)."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
TYPES = ("float32", "bfloat16", "float16")
ROWS = (1, 2, 3, 4, 5, 16, 17, 40)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [20, 31, 33, 64, 96, 100, 127, 128, 130, 160, 224, 500, 2048 + 33, 4128])
def test_scales_that_are_not_finite(k, dtype):
    """Positive activations and codes above the zero point: each sum of a group is positive, and
    the output is its scale's infinity or NaN, whichever group has it."""
    t = torch()
    group, n = 32, 37
    groups = -(-k // group)
    gen = t.Generator().manual_seed(k)
    q = t.randint(9, 16, (n, (k + 1) // 2), generator=gen, dtype=t.uint8)
    q = (q | (t.randint(9, 16, q.shape, generator=gen, dtype=t.uint8) << 4)).cuda()
    for at in (0, groups - 1):
        for stype in TYPES:
            s = t.full((n, groups), 0.5, dtype=getattr(t, stype), device="cuda")
            s[3, at], s[4, at], s[20, at], s[36, at] = float("inf"), float("-inf"), float("nan"), float("inf")
            for m in ROWS:
                a = (t.rand((m, k), generator=gen) + 0.5).to(getattr(t, dtype)).cuda()
                say(f"q4 {m}x{n}x{k} {dtype} scales {stype} group {at}")
                out = og.gemm_nt_q4(a, q, s, group=group)
                special = [3, 4, 20, 36]
                assert (out[:, [3, 36]] == float("inf")).all() and (out[:, 4] == float("-inf")).all()
                assert out[:, 20].isnan().all()
                rest = [j for j in range(n) if j not in special]
                exact, bound = ref.q4(a, q[rest], s[rest], None, group)
                assert ((out[:, rest].double() - exact).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", ROWS)
def test_scales_multiply_sums_of_32(m, dtype):
    """Activations and codes with zeros, signs and sums of zero among them: infinite scales give
    what they give times each sum of 32 terms.  Whole numbers below 2^12 times a half: the finite
    results are exact in fp32 and rounded once."""
    t = torch()
    n, k, group = 50, 320, 64
    gen = t.Generator().manual_seed(m)
    q = t.randint(0, 256, (n, k // 2), generator=gen, dtype=t.uint8).cuda()
    a = t.randint(-1, 2, (m, k), generator=gen).to(getattr(t, dtype)).cuda()
    a[:, 96:128] = 0
    s = t.full((n, k // group), 0.5, device="cuda")
    s[::3, 0], s[1::5, 1], s[2::7, 4], s[::11, 4] = float("inf"), float("-inf"), float("inf"), float("-inf")
    sums = (ref.q4_weights(q, t.ones_like(s), None, k, group)[None] * a.double()[:, None]).view(m, n, k // 32, 32).sum(3)
    want = (sums * s.double().repeat_interleave(2, 1)[None]).sum(2)
    say(f"q4 {m}x{n}x{k} {dtype}")
    out = og.gemm_nt_q4(a, q, s, group=group).double()
    assert want.isinf().any() and want.isnan().any()
    assert t.equal(out.isnan(), want.isnan())
    inf = want.isinf()
    assert t.equal(out[inf], want[inf])
    fin = want.isfinite()
    assert ((out - want).abs()[fin] <= ref.half_step(getattr(t, dtype)) * want.abs()[fin]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", ROWS)
def test_activations_that_are_not_finite(m, dtype):
    t = torch()
    n, k, group = 40, 320, 64
    gen = t.Generator().manual_seed(m)
    q = t.randint(0, 256, (n, k // 2), generator=gen, dtype=t.uint8).cuda()
    s = (t.rand((n, k // group), generator=gen) + 0.1).cuda()
    w = ref.q4_weights(q, s, None, k, group)
    for value in (float("inf"), float("-inf"), float("nan")):
        for p in (0, 77, 319):
            a = t.randn((m, k), generator=gen).to(getattr(t, dtype)).cuda()
            a[m // 2, p] = value
            say(f"q4 {m}x{n}x{k} {dtype} {value} at {p}")
            out = og.gemm_nt_q4(a, q, s, group=group).double()
            want = t.where(w[:, p] == 0, t.nan, t.sign(w[:, p]) * value)
            assert t.equal(out[m // 2].isnan(), want.isnan())
            assert t.equal(out[m // 2].nan_to_num(nan=1.0), want.nan_to_num(nan=1.0))
            rest = [i for i in range(m) if i != m // 2]
            exact, bound = ref.q4(a[rest], q, s, None, group)
            assert ((out[rest] - exact).abs() <= bound).all()


@pytest.mark.parametrize("m", ROWS)
def test_the_largest_fp32_activations(m):
    """Values past the largest bf16 (up to the largest fp32) times 1 or -1, halved by the scale."""
    t = torch()
    n, k, group = 20, 160, 32
    q = t.full((n, k // 2), 0x99, dtype=t.uint8, device="cuda")
    q[1::2] = 0x77
    s = t.full((n, k // group), 0.5, device="cuda")
    top = t.finfo(t.float32).max
    for p, value in ((0, top), (33, -top), (159, 3.39e38), (64, 3.3961775e38), (65, -3.4e38)):
        a = t.zeros((m, k), device="cuda")
        a[:, p] = value
        say(f"q4 {m}x{n}x{k} {value} at {p}")
        out = og.gemm_nt_q4(a, q, s, group=group)
        exact, bound = ref.q4(a, q, s, None, group)
        assert ((out.double() - exact).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", ROWS)
def test_every_code_and_zero_point(m, dtype):
    """All sixteen codes against all zero points a byte can hold, whole numbers: exact."""
    t = torch()
    q = (t.arange(16, dtype=t.uint8)[:, None] * 17).repeat(16, 16).cuda()  # row j: code j % 16
    s = t.full((256, 1), 0.5, device="cuda")
    say(f"q4 {m} rows {dtype}")
    for first in range(0, 256, 16):
        z = t.arange(first, first + 16, dtype=t.uint8).repeat_interleave(16)[:, None].cuda()
        a = t.zeros((m, 32), dtype=getattr(t, dtype), device="cuda")
        a[:, 7], a[:, 30] = 3, -1
        out = og.gemm_nt_q4(a, q, s, zeros=z, group=32)
        want = (q[:, 0] % 16).double() - z[:, 0].double()
        # (at most 8 bits: every type holds them)
        assert t.equal(out.double(), want.expand(m, 256)), first
