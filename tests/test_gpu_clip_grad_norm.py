"""og_grad_norm and og_clip_grad_norm against 64 bits: types mixed, many tensors, odd sizes and
offsets, strides, values whose squares leave fp32's range, values that are not finite, in place."""
import math

import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
EVERY = ("float32", "bfloat16", "float16")


def tensors(shapes, types, seed=0, scale=1.0):
    th = torch()
    gen = th.Generator().manual_seed(seed)
    return [(scale * th.randn(s, generator=gen)).to(getattr(th, types[i % len(types)])).cuda()
            for i, s in enumerate(shapes)]


def exact_norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check(grads, got, norm, max_norm, eps):
    """The norm: squares are exact, sums in 64 bits, one rounding.  A result: the factor's
    rounding and the product's (2^-24 each), then the type's (half a step, or of its smallest)."""
    th = torch()
    want = exact_norm(grads)
    assert abs(float(norm) - want) <= 2.0 ** -24 * 1.001 * want
    by = min(1.0, max_norm / (want + eps)) if want + eps > 0 else 1.0
    for g, y in zip(grads, got):
        x = g.double() * by
        e = x.abs() * 2.0 ** -23 * 1.01
        tiny = th.finfo(g.dtype).smallest_normal * th.finfo(g.dtype).eps
        assert ((y.double() - x).abs() <= e + ref.half_step(g.dtype) * (x.abs() + e) + tiny).all()
        if by == 1.0:
            assert th.equal(y, g)


SHAPES = {"one": [(1,)], "odd": [(3, 5), (17,), (1,), (1023,), (129, 257), (4, 3, 2, 5)],
          "empty among": [(0,), (7, 0), (33,), (0, 4), (5, 5)], "chunk": [(8192,), (4096,), (4097,), (8191,), (65536,)],
          "large": [(1100, 3000), (500001,), (2048, 1024)], "many": [(i % 37 + 1, i % 11 + 1) for i in range(333)]}


@pytest.mark.parametrize("types", [(t,) for t in EVERY] + [EVERY])
@pytest.mark.parametrize("name", list(SHAPES))
def test_clip(name, types):
    th = torch()
    grads = tensors(SHAPES[name], types)
    for max_norm in (1.0, 1e9):
        say(f"clip_grad_norm {name} {types} {max_norm}")
        out = [th.full_like(g, 7.0) for g in grads]
        norm = og.clip_grad_norm(grads, max_norm, eps=1e-6, out=out)
        check(grads, out, norm, max_norm, 1e-6)
        mine = [g.clone() for g in grads]
        again = og.clip_grad_norm(mine, max_norm, eps=1e-6)
        assert th.equal(norm, again) and all(th.equal(a, b) for a, b in zip(mine, out))
        assert th.equal(og.grad_norm(grads), norm)


@pytest.mark.parametrize("dtype", EVERY)
@pytest.mark.parametrize("first", [0, 1, 3, 8])
def test_views_of_one_buffer(first, dtype):
    """Gradients as parts of one flat buffer, at any offset; nothing between them is written."""
    th = torch()
    flat = tensors([(70000,)], (dtype,), seed=first)[0]
    was = flat.clone()
    parts, at = [], first
    for size in (1, 5000, 16384, 33, 20001):
        parts.append((at, at + size))
        at += size + 2
    norm = og.clip_grad_norm([flat[a:b] for a, b in parts], 0.5)
    check([was[a:b] for a, b in parts], [flat[a:b] for a, b in parts], norm, 0.5, 1e-6)
    keep = th.ones_like(flat, dtype=th.bool)
    for a, b in parts:
        keep[a:b] = False
    assert th.equal(flat[keep], was[keep])


@pytest.mark.parametrize("dtype", EVERY)
def test_strides(dtype):
    """Column slices of one matrix, transposed matrices, single rows and columns, channels of
    an image tensor in any dense order."""
    th = torch()
    w = tensors([(300, 500)], (dtype,))[0]
    was = w.clone()
    cuts = [(0, 200), (200, 201), (203, 500)]
    norm = og.clip_grad_norm([w[:, a:b] for a, b in cuts], 3.0)
    check([was[:, a:b] for a, b in cuts], [w[:, a:b] for a, b in cuts], norm, 3.0, 1e-6)
    assert th.equal(w[:, 201:203], was[:, 201:203])
    views = [was.t(), was[7:8, 3:90], was[::2, :100], was[:, :1]]
    out = [th.empty_like(v) for v in views]
    out[0] = th.empty((300, 500), dtype=w.dtype, device="cuda").t()
    norm = og.clip_grad_norm(views, 3.0, out=out)
    check(views, out, norm, 3.0, 1e-6)
    # from a slice to a contiguous tensor and back
    out = [th.empty((300, 200), dtype=w.dtype, device="cuda"), w[:, 250:450]]
    norm = og.clip_grad_norm([was[:, :200], was[:, 100:300].contiguous()], 3.0, out=out)
    check([was[:, :200], was[:, 100:300]], out, norm, 3.0, 1e-6)


@pytest.mark.parametrize("dtype", EVERY)
def test_dense_in_any_order(dtype):
    """Convolution weights with the channels last, permuted tensors, single elements of any stride;
    a slice of one is refused and nothing is written."""
    th = torch()
    flat = tensors([(24 * 5 * 3 * 3,)], (dtype,))[0]
    views = [flat.view(24, 3, 3, 5).permute(0, 3, 1, 2), tensors([(7, 6, 5)], (dtype,))[0].permute(2, 0, 1),
             tensors([(9, 4)], (dtype,))[0][3:4, 1:2], tensors([(9, 4)], (dtype,))[0][:, 2:3]]
    was = [v.clone() for v in views]
    out = [th.empty_like(v) for v in views]
    assert out[0].stride() == views[0].stride()
    check(was, out, og.clip_grad_norm(views, 0.7, out=out), 0.7, 1e-6)
    check(was, views, og.clip_grad_norm(views, 0.7), 0.7, 1e-6)
    kept = flat.clone()
    with pytest.raises(ValueError):
        og.clip_grad_norm([views[0][:, :4]], 0.1)
    assert th.equal(flat, kept)


@pytest.mark.parametrize("scale", [1e30, 1e-30, 3e-39])
def test_range(scale):
    """Squares outside fp32's range, subnormal values."""
    grads = tensors([(1000,), (37, 91)], ("float32", "bfloat16"), scale=scale)
    for max_norm in (1.0, 1e-30):
        out = [torch().empty_like(g) for g in grads]
        check(grads, out, og.clip_grad_norm(grads, max_norm, eps=0.0, out=out), max_norm, 0.0)


def test_zeros_and_limits():
    th = torch()
    zeros = [th.zeros(100, device="cuda"), th.zeros((3, 4), device="cuda").half()]
    for max_norm, eps in ((1.0, 1e-6), (0.0, 0.0), (0.0, 1e-6), (1.0, 0.0)):
        got = [z.clone() for z in zeros]
        assert og.clip_grad_norm(got, max_norm, eps=eps) == 0
        assert all((g == 0).all() for g in got)
    ones = [th.ones(16, device="cuda")]
    assert og.clip_grad_norm(ones, 0.0) == 4 and (ones[0] == 0).all()


@pytest.mark.parametrize("dtype", EVERY)
def test_not_finite(dtype):
    """An infinite norm: finite elements 0, infinite ones NaN; a NaN norm: NaN."""
    th = torch()
    for bad in (float("inf"), float("-inf"), float("nan")):
        grads = tensors([(100,), (5000,)], (dtype,))
        grads[1][4321] = bad
        norm = og.clip_grad_norm(grads, 1.0)
        if bad == bad:
            assert norm == float("inf")
            assert (grads[0] == 0).all() and grads[1][4321].isnan() and (grads[1][:4321] == 0).all()
        else:
            assert norm.isnan() and all(g.isnan().all() for g in grads)


def test_repeats_bit_for_bit_and_workspace():
    th = torch()
    grads = tensors([(777, 333), (100000,), (13,)], EVERY, seed=3)
    size = og.lib().og_grad_norm_workspace()
    whole = th.full((size + 512,), 0xA5, dtype=th.uint8, device="cuda")
    want = og.grad_norm(grads)
    for byte in (0, 0xFF, 0x7B):
        whole[256:256 + size].fill_(byte)
        assert th.equal(og.grad_norm(grads, workspace=whole[256:256 + size]), want)
    assert (whole[:256] == 0xA5).all() and (whole[256 + size:] == 0xA5).all()
    with pytest.raises(og.OgError):
        og.grad_norm(grads, workspace=whole[:size - 1])


def test_refused_by_the_binding():
    th = torch()
    a, b = th.ones((4, 6), device="cuda"), th.ones(5, device="cuda")
    for grads, kw in [([], {}), ([a, a.double()], {}), ([a, b.cpu()], {}), ([a.cpu()], {}), ([a[:, ::2]], {}),
                      ([a.expand(3, 4, 6)], {}), ([a], dict(out=[])), ([a], dict(out=[b])),
                      ([a], dict(out=[a.half()])), ([a], dict(out=[th.ones((6, 4), device="cuda").t()]))]:
        with pytest.raises(ValueError):
            og.clip_grad_norm(grads, 1.0, **kw)
    for grads, limit, eps in [([a], -1.0, 1e-6), ([a], float("nan"), 1e-6), ([a], float("inf"), 1e-6),
                              ([a], 1.0, -1e-6), ([a], 1.0, float("nan")), ([a, b, a], 1.0, 1e-6)]:
        with pytest.raises(og.OgError):
            og.clip_grad_norm(grads, limit, eps=eps)
    assert (a == 1).all() and (b == 1).all()
