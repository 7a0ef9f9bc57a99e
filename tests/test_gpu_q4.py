"""The product with 4-bit weights against its definition in 64 bits."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
TYPES = ("float32", "bfloat16", "float16")


def make(m, n, k, group, dtype, stype="float32", zeros=True, seed=0):
    t = torch()
    gen = t.Generator().manual_seed(seed)
    groups = -(-k // group)
    a = t.randn((m, k), generator=gen).to(getattr(t, dtype)).cuda()
    q = t.randint(0, 256, (n, (k + 1) // 2), generator=gen, dtype=t.uint8).cuda()
    s = (t.rand((n, groups), generator=gen) * 0.02 + 0.001).to(getattr(t, stype)).cuda()
    z = t.randint(0, 16, (n, groups), generator=gen, dtype=t.uint8).cuda() if zeros else None
    return a, q, s, z


def check(out, a, q, s, z, group, what):
    t = torch()
    exact, bound = ref.q4(a, q, s, z, group)
    off = (out.double() - exact).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {off.numel()} outputs off by up to "
                           f"{float((off / bound)[bad].max()):.3g} times the bound")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,group", [
    (1, 1, 1, 32), (1, 16, 128, 128), (1, 17, 127, 64), (2, 5, 33, 32), (3, 100, 31, 32),
    (16, 64, 2048, 128), (17, 33, 2049, 32), (1, 1000, 4097, 96), (33, 48, 640, 256),
    (5, 70, 1000, 4096), (1, 4096, 4096, 128), (100, 129, 300, 32), (64, 300, 515, 160),
])
def test_shapes(m, n, k, group, dtype):
    for zeros, stype in ((True, "float32"), (False, "float16"), (True, "bfloat16")):
        a, q, s, z = make(m, n, k, group, dtype, stype, zeros, seed=m * n + k)
        say(f"q4 {m}x{n}x{k} group {group} {dtype} scales {stype} zeros {zeros}")
        check(og.gemm_nt_q4(a, q, s, zeros=z, group=group), a, q, s, z, group, (m, n, k))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 16, 17, 40])
def test_lengths_around_a_load_and_wide_layers(m, dtype):
    """k around the 32 codes of a load and where a row's pieces divide among the waves; weights
    enough for two tiles of rows a block."""
    for n, k in ((70, 30), (70, 31), (70, 32), (70, 33), (9, 2047), (9, 4128), (9, 8193), (8200, 95),
                 (8250, 256)):
        a, q, s, z = make(m, n, k, 32, dtype, seed=m + n + k)
        say(f"q4 {m}x{n}x{k} {dtype}")
        check(og.gemm_nt_q4(a, q, s, zeros=z, group=32), a, q, s, z, 32, (m, n, k))


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_offsets_and_gaps(dtype):
    """Row strides, odd byte offsets of the codes, a NaN sentinel in every gap of the inputs
    and one in the output's that must survive."""
    t = torch()
    m, n, k, group = 5, 37, 301, 32
    a, q, s, z = make(m, n, k, group, dtype, seed=5)
    big_a = t.full((m, k + 13), float("nan"), dtype=a.dtype, device="cuda")
    big_a[:, 3:3 + k] = a
    big_q = t.full((n, q.shape[1] + 7), 255, dtype=t.uint8, device="cuda")
    big_q[:, 1:1 + q.shape[1]] = q
    big_s = t.full((n, s.shape[1] + 3), float("nan"), device="cuda")
    big_s[:, 1:1 + s.shape[1]] = s
    big_z = t.full((n, s.shape[1] + 5), 99, dtype=t.uint8, device="cuda")
    big_z[:, 2:2 + s.shape[1]] = z
    big_c = t.full((m, n + 9), 7.5, dtype=a.dtype, device="cuda")
    og.gemm_nt_q4(big_a[:, 3:3 + k], big_q[:, 1:1 + q.shape[1]], big_s[:, 1:1 + s.shape[1]],
                  zeros=big_z[:, 2:2 + s.shape[1]], group=group, out=big_c[:, 4:4 + n])
    check(big_c[:, 4:4 + n], a, q, s, z, group, "strided")
    assert (big_c[:, :4] == 7.5).all() and (big_c[:, 4 + n:] == 7.5).all()


def test_codes_at_the_end_of_an_allocation():
    """The last row's codes end with the allocation, at every remainder of 16 bytes."""
    t = torch()
    for k in range(1, 70, 3):
        a, q, s, z = make(2, 3, k, 32, "float32", seed=k)
        flat = t.zeros(q.numel() + 5, dtype=t.uint8, device="cuda")
        tail = flat[5:].view(q.shape)
        tail.copy_(q)
        check(og.gemm_nt_q4(a, tail, s, zeros=z, group=32), a, q, s, z, 32, k)


def test_k_zero_and_empty():
    t = torch()
    a = t.ones((3, 0), device="cuda")
    q = t.ones((4, 0), dtype=t.uint8, device="cuda")
    s = t.ones((4, 0), device="cuda")
    assert (og.gemm_nt_q4(a, q, s, group=32) == 0).all()
    a, q, s, z = make(1, 4, 64, 32, "bfloat16")
    assert og.gemm_nt_q4(a[:0], q, s, zeros=z, group=32).shape == (0, 4)
    assert og.gemm_nt_q4(a, q[:0], s[:0], zeros=z[:0], group=32).shape == (1, 0)


@pytest.mark.parametrize("dtype", TYPES)
def test_special_activations(dtype):
    """Infinities and NaN act as in the formula; a row's large value does not cost its other
    slices or rows their bits; rows of zeros and of tiny values."""
    t = torch()
    m, n, k, group = 9, 40, 512, 32
    a, q, s, z = make(m, n, k, group, dtype, seed=9)
    a[0, 5] = float("inf")
    a[1, 500] = float("-inf")
    a[2, 77] = float("nan")
    a[3, :] = 0
    a[4, 3] = 60000.0
    if dtype != "float16":
        a[5] *= 2.0 ** -120
        a[6] *= 2.0 ** 100
        a[7, 10] = 2.0 ** 120
    out = og.gemm_nt_q4(a, q, s, zeros=z, group=group).double()
    w = ref.q4_weights(q, s, z, k, group)
    for i, p in ((0, 5), (1, 500)):
        want = t.where(w[:, p] == 0, t.nan, t.sign(w[:, p]) * a[i, p].double())
        assert t.equal(t.nan_to_num(out[i], nan=1.0), t.nan_to_num(want, nan=1.0)), i
        assert t.equal(out[i].isnan(), want.isnan())
    assert out[2].isnan().all()
    rest = [3, 4, 5, 6, 7, 8]
    check(og.gemm_nt_q4(a, q, s, zeros=z, group=group)[rest], a[rest], q, s, z, group, "special")
    assert (out[3] == 0).all()


def test_every_code_and_zero_point():
    """All sixteen codes against all zero points a byte can hold, whole numbers: exact."""
    t = torch()
    q = (t.arange(16, dtype=t.uint8)[:, None] * 17).repeat(16, 16).cuda()  # row j: code j % 16
    for first in range(0, 256, 16):
        z = t.arange(first, first + 16, dtype=t.uint8).repeat_interleave(16)[:, None].cuda()
        s = t.full((256, 1), 0.5, device="cuda")
        for dtype in TYPES:
            a = t.zeros((1, 32), dtype=getattr(t, dtype), device="cuda")
            a[0, 7], a[0, 30] = 3, -1
            out = og.gemm_nt_q4(a, q, s, zeros=z, group=32)
            want = (q[:, 0] % 16).double() - z[:, 0].double()
            assert t.equal(out[0].double(), want), (first, dtype)


def test_long_rows_past_32_bits():
    """Row offsets of the codes past 2^32 bytes: the last rows of a matrix with a long stride."""
    t = torch()
    a, q, s, z = make(1, 48, 256, 64, "bfloat16", seed=3)
    stride = 100 << 20
    flat = t.empty(47 * stride + q.shape[1], dtype=t.uint8, device="cuda")
    view = t.as_strided(flat, q.shape, (stride, 1))
    view.copy_(q)
    check(og.gemm_nt_q4(a, view, s, zeros=z, group=64), a, q, s, z, 64, "long rows")
