"""og_gemm_nt_epi and its gradient against 64 bits: types, activations, sizes from one to some
thousands, odd ones, strides and offsets, special values, rows of all sizes, what is not written."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
EVERY = ("float32", "bfloat16", "float16")
ACTS = (None, "relu", "gelu", "gelu_tanh", "silu")


def make(m, n, k, dtype, seed=0, bias=True, residual=True):
    th = torch()
    gen = th.Generator().manual_seed(seed + m + 3 * n + 7 * k)
    kind = getattr(th, dtype)
    rnd = lambda *s: th.randn(s, generator=gen)  # noqa: E731
    c = dict(A=rnd(m, k), B=rnd(n, k) / max(k, 1) ** 0.5, bias=rnd(n) if bias else None,
             residual=rnd(m, n) if residual else None)
    c = {name: None if t is None else t.to(kind).cuda() for name, t in c.items()}
    dc = rnd(m, n).to(kind).cuda()
    if m:
        dc[m // 2] = 0
    return c, dc


def inside(got, want, bound):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), (off / bound).nan_to_num(nan=float("inf")).max().item()


def check_forward(c, act, got, pre=None):
    e = ref.gemm_epi(c["A"], c["B"], c["bias"], act, c["residual"])
    inside(got, e["c"], e["e_c"])
    if pre is not None:
        inside(pre, e["pre"], e["e_pre"])


def check_grad(c, dc, pre, act, got):
    e = ref.gemm_epi_grad(dc, c["A"], c["B"], pre, act)
    for name, t in zip(("da", "dw", "dbias"), got):
        if t is not None:
            say(name)
            inside(t, e[name], e["e_" + name])


SIZES = [(1, 1, 1), (1, 5, 3), (1, 33, 70), (2, 64, 128), (3, 100, 257), (5, 16, 1000), (16, 130, 520), (17, 31, 33),
         (33, 257, 40), (64, 64, 64), (65, 200, 1), (70, 1, 300), (129, 131, 100), (200, 777, 96), (300, 256, 512),
         (1000, 120, 61), (513, 520, 1030)]


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_sizes(m, n, k, dtype):
    for i, act in enumerate(ACTS):
        c, dc = make(m, n, k, dtype, seed=i, bias=i != 1, residual=i % 2 == 0)
        say(f"gemm_nt_epi {m}x{n}x{k} {dtype} {act}")
        out, pre = og.gemm_nt_epi(**c, act=act, need_pre=True)
        check_forward(c, act, out, pre)
        assert torch().equal(og.gemm_nt_epi(**c, act=act), out)
        say(f"gemm_nt_epi_grad {m}x{n}x{k} {dtype} {act}")
        got = og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act=act)
        check_grad(c, dc, pre, act, got)


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (16, 4096, 1100), (40, 2000, 4100), (777, 1531, 1000),
                                   (2048, 512, 768), (1100, 4096, 300)])
def test_larger(m, n, k, dtype):
    c, dc = make(m, n, k, dtype, seed=5, residual=False)
    say(f"gemm_nt_epi {m}x{n}x{k} {dtype}")
    out, pre = og.gemm_nt_epi(**c, act="gelu", need_pre=True)
    check_forward(c, "gelu", out, pre)
    check_grad(c, dc, pre, "gelu", og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act="gelu"))


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("m,n,k", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0), (300, 40, 0), (0, 300, 64), (70, 0, 64)])
def test_empty(m, n, k, dtype):
    th = torch()
    c, dc = make(m, n, k, dtype)
    say(f"gemm_nt_epi {m}x{n}x{k} {dtype}")
    out, pre = og.gemm_nt_epi(**c, act="silu", need_pre=True)
    check_forward(c, "silu", out, pre)
    got = [th.full(s, 3.0, dtype=dc.dtype, device="cuda") for s in ((m, k), (n, k), (n,))]
    og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act="silu", dA=got[0], dB=got[1], dbias=got[2])
    check_grad(c, dc, pre, "silu", got)


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("m,n,k", [(3, 100, 64), (20, 72, 130), (150, 200, 256), (129, 96, 77)])
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_strides(m, n, k, offset, dtype):
    """Every matrix inside a wider one, at an offset: results as of contiguous ones, nothing
    beside them written; the residual in the output's place."""
    th = torch()
    c, dc = make(m, n, k, dtype, seed=offset)
    say(f"gemm_nt_epi strides {m}x{n}x{k}+{offset} {dtype}")

    def wide(t, pad=24):
        w = th.full((t.shape[0], t.shape[1] + pad), 1e3, dtype=t.dtype, device="cuda")
        v = w[:, offset:offset + t.shape[1]]
        v.copy_(t)
        return w, v

    def untouched(w, v):
        v.fill_(1e3)
        return bool((w == 1e3).all())

    A, B, (wr, R), (_, D) = wide(c["A"])[1], wide(c["B"])[1], wide(c["residual"]), wide(dc)
    wp, P = wide(c["residual"])
    bias = th.cat([c["bias"][:1], c["bias"]])[1:]
    want, pre = og.gemm_nt_epi(**c, act="gelu_tanh", need_pre=True)
    got, _ = og.gemm_nt_epi(A, B, bias=bias, act="gelu_tanh", residual=R, out=R, pre=P)
    assert got is R and th.equal(R, want) and th.equal(P, pre)
    grads = og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act="gelu_tanh")
    check_grad(c, dc, pre, "gelu_tanh", grads)
    (wa, dA), (wb, dB) = wide(c["A"]), wide(c["B"])
    og.gemm_nt_epi_grad(D, A, B, pre=P, act="gelu_tanh", dA=dA, dB=dB)
    assert th.equal(dA, grads[0]) and th.equal(dB, grads[1])
    assert untouched(wr, R) and untouched(wp, P) and untouched(wa, dA) and untouched(wb, dB)


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("act", [None, "silu"])
def test_parts_of_the_gradient(act, dtype):
    th = torch()
    c, dc = make(130, 96, 200, dtype)
    _, pre = og.gemm_nt_epi(**c, act=act, need_pre=True)
    every = og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act=act)
    for need in [(True, False, False), (False, True, False), (False, False, True), (True, False, True),
                 (False, True, True), (True, True, False), (False, False, False)]:
        got = og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act=act, need=need)
        for a, b, wanted in zip(got, every, need):
            assert (a is None) if not wanted else th.equal(a, b)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", EVERY)
def test_activations_over_their_range(act, dtype):
    """v is the bias alone where A is zero: the activation and its slope from far left to far right."""
    th = torch()
    kind = getattr(th, dtype)
    x = th.cat([th.linspace(-130, 130, 3001), th.linspace(-9, 9, 2000), th.logspace(-30, 4, 500),
                -th.logspace(-30, 4, 500)]).to(kind).cuda()
    n = len(x)
    A, B = th.zeros((2, 8), dtype=kind, device="cuda"), th.ones((n, 8), dtype=kind, device="cuda")
    out, pre = og.gemm_nt_epi(A, B, bias=x, act=act, need_pre=True)
    assert th.equal(pre[0], x) and th.equal(pre[1], x)
    check_forward(dict(A=A, B=B, bias=x, residual=None), act, out)
    dc = th.ones((1, n), dtype=kind, device="cuda")
    got = og.gemm_nt_epi_grad(dc, A[:1], B, pre=pre[:1], act=act, need=(False, False, True))
    check_grad(dict(A=A[:1], B=B), dc, pre[:1], act, got)


@pytest.mark.parametrize("m", [1, 3, 40, 200])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", EVERY)
def test_infinities_and_nan(act, dtype, m):
    """In the bias and the residual every type follows the formula; 16-bit ones in A and W too."""
    th = torch()
    inf, nan = float("inf"), float("nan")
    c, _ = make(m, 64, 96, dtype)
    c["bias"][:4] = th.tensor([inf, -inf, nan, 5.0], device="cuda")
    c["residual"][0, 5:8] = th.tensor([inf, -inf, nan], device="cuda")
    if dtype != "float32":
        c["A"][0, 3] = 0
        c["B"][10, 3], c["B"][11, 5], c["B"][12, 7] = inf, inf, nan
    out, pre = og.gemm_nt_epi(**c, act=act, need_pre=True)
    v = c["A"].double().cpu() @ c["B"].double().cpu().t() + c["bias"].double().cpu()
    y = ref.activation(v, act)[0] + c["residual"].double().cpu()
    for got, want in ((pre, v), (out, y)):
        got = got.double().cpu()
        assert th.equal(got.isnan(), want.isnan())
        assert th.equal(got[want.isinf()], want[want.isinf()]) and th.equal(got.isinf(), want.isinf())
    dc = th.ones_like(out)
    db = og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act=act, need=(False, False, True))[2].double().cpu()
    want = ref.activation(pre.double().cpu(), act)[1].sum(0)
    assert th.equal(db.isnan(), want.isnan()) and not db.isinf().any()


@pytest.mark.parametrize("m", [2, 150])
def test_fp32_rows_of_all_sizes(m):
    """Every row of A and W, and every row and column of the gradients' operands, to its own size."""
    th = torch()
    n, k = 150, 160
    c, dc = make(m, n, k, "float32", bias=False, residual=False)
    powers = lambda count: (2.0 ** th.linspace(-60, 55, count).round()).cuda()  # noqa: E731
    c["A"] *= powers(m)[:, None]
    c["B"] *= powers(n).flip(0)[:, None]
    c["A"][m // 2] = 0
    c["B"][5] = 0
    out = og.gemm_nt_epi(**c)
    check_forward(c, None, out)
    assert (out[m // 2] == 0).all() and (out[:, 5] == 0).all()
    # dA: rows of dC and columns of W differ; dW: columns of dC and of A
    c, dc = make(m, n, k, "float32")
    dc2 = dc * powers(m)[:, None]
    c["B"] *= powers(k)[None]
    check_grad(c, dc2, None, None, og.gemm_nt_epi_grad(dc2, c["A"], c["B"], need=(True, False, False)))
    dc3 = dc * powers(n)[None]
    c["A"] *= powers(k)[None]
    dc3[:, 7] = 0
    check_grad(c, dc3, None, None, og.gemm_nt_epi_grad(dc3, c["A"], c["B"], need=(False, True, True)))


def test_fp16_gradients_at_the_ends_of_the_range():
    """A dC near the largest fp16 times a slope above 1, and subnormal ones."""
    th = torch()
    m, n, k = 70, 64, 64
    c, dc = make(m, n, k, "float16")
    c["B"] *= 1e-4
    dc.fill_(65000.0)
    pre = th.full((m, n), 1.5, device="cuda").half()
    got = og.gemm_nt_epi_grad(dc, c["A"] * 1e-4, c["B"], pre=pre, act="gelu", need=(True, True, False))
    check_grad(dict(A=c["A"] * 1e-4, B=c["B"]), dc, pre, "gelu", got)
    c, dc = make(m, n, k, "float16")
    dc *= 1e-6
    c["B"] *= 100
    check_grad(c, dc, pre, "silu", og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act="silu"))


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
def test_gradient_against_differences(act, dtype):
    """The gradients of sum(C * dC) against central differences of the 64-bit formula."""
    th = torch()
    c, dc = make(20, 24, 32, dtype, residual=False)
    _, pre = og.gemm_nt_epi(**c, act=act, need_pre=True)
    got = og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act=act)
    a, w, b = (c[x].double() for x in ("A", "B", "bias"))

    def f(a, w, b):
        return (ref.activation(a @ w.t() + b, act)[0] * dc.double()).sum()

    gen = th.Generator(device="cuda").manual_seed(1)
    for i, (t, g) in enumerate(zip((a, w, b), got)):
        d = th.randn(t.shape, generator=gen, device="cuda", dtype=th.float64)
        h = 1e-5
        args = [[x + h * s * d if j == i else x for j, x in enumerate((a, w, b))] for s in (1, -1)]
        slope = (f(*args[0]) - f(*args[1])) / (2 * h)
        # each element's error: dP's and the result's rounding and P's (its slope changes by 0.8 of that at
        # most), all of one step of the type; the sums of their sizes along d
        size = ((dc.double().abs().t() @ a.abs()) if i == 1 else (dc.double().abs() @ w.abs()) if i == 0
                else dc.double().abs().sum(0))
        bound = (size * d.abs()).sum() * (4 * STEP[dtype] * (1 + pre.double().abs().max())) + 1e-6
        assert (g.double() * d).sum().sub(slope).abs() <= bound


STEP = {"float32": 2.0 ** -20, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


def test_refused_by_the_binding():
    th = torch()
    c, dc = make(4, 6, 8, "float32")
    A, B = c["A"], c["B"]
    for args, kw in [((A, B[:, :7]), {}), ((A, B.half()), {}), ((A.double(), B.double()), {}), ((A[0], B), {}),
                     ((A, B), dict(act="tanh")), ((A, B), dict(bias=c["bias"][:5])),
                     ((A, B), dict(bias=c["bias"].half())), ((A, B), dict(residual=c["residual"][:3])),
                     ((A, B), dict(out=dc.half())), ((A, B), dict(pre=dc[:, :5])), ((A, B.cpu()), {}),
                     ((A, B), dict(residual=c["residual"].t().contiguous().t()))]:
        with pytest.raises(ValueError):
            og.gemm_nt_epi(*args, **kw)
    with pytest.raises(og.OgError):
        og.gemm_nt_epi(A, B, residual=c["residual"][:1].expand(4, 6))
    with pytest.raises(og.OgError):
        og.gemm_nt_epi(A, B, out=dc, pre=dc)
    for kw in [dict(act="gelu"), dict(act="gelu", pre=dc[:3]), dict(dA=B), dict(dB=A), dict(dbias=c["bias"][:2])]:
        with pytest.raises(ValueError):
            og.gemm_nt_epi_grad(dc, A, B, **kw)
    with pytest.raises(ValueError):
        og.gemm_nt_epi_grad(dc[:3], A, B)


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("m,n,k", [(1100000, 1, 1), (1100000, 2, 0), (90000, 3, 5), (2, 70000, 3)])
def test_many_rows(m, n, k, dtype):
    """More row blocks than a launch's second axis has."""
    c, dc = make(m, n, k, dtype)
    say(f"gemm_nt_epi {m}x{n}x{k} {dtype}")
    out, pre = og.gemm_nt_epi(**c, act="relu", need_pre=True)
    check_forward(c, "relu", out, pre)
    check_grad(c, dc, pre, "relu", og.gemm_nt_epi_grad(dc, c["A"], c["B"], pre=pre, act="relu"))


def test_outputs_past_32_bits():
    """C, P and dC of more than 4 GiB: the last rows, and the gradient that they enter."""
    th = torch()
    m, n, k = 66000, 33024, 64
    gen = th.Generator(device="cuda").manual_seed(0)
    A = th.randn((m, k), generator=gen, device="cuda").bfloat16()
    B = (0.1 * th.randn((n, k), generator=gen, device="cuda")).bfloat16()
    say(f"gemm_nt_epi {m}x{n}x{k}")
    out, pre = og.gemm_nt_epi(A, B, act="silu", need_pre=True)
    e = ref.gemm_epi(A[-70:], B, None, "silu", None)
    inside(out[-70:], e["c"], e["e_c"])
    inside(pre[-70:], e["pre"], e["e_pre"])
    dA = og.gemm_nt_epi_grad(out, A, B, pre=pre, act="silu", need=(True, False, False))[0]
    # (of more than 128 rows: dP is rounded to the type once)
    wide = th.cat([out[-70:], out[-70:]]), th.cat([A[-70:], A[-70:]]), th.cat([pre[-70:], pre[-70:]])
    e = ref.gemm_epi_grad(wide[0], wide[1], B, wide[2], "silu")
    inside(dA[-70:], e["da"][:70], e["e_da"][:70])
