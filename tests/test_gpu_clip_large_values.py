"""og_clip_grad_norm at the top of fp32's and bf16's range: elements and norms past half of the largest
value, and a norm that only 64 bits hold."""
import math

import pytest

import fp32_blocked_gemm_amd as og
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
TOP = 2.0 ** 127
# elements as multiples of 2^127; the largest fp32 is just below 2, the largest bf16 1.9921875
VALUES = {"one": [1.5], "largest": [1.9921875], "with small ones": [1.0, -1.75, 1e-38, 1e-30, 0.0],
          "norm past fp32": [1.75, 1.75], "many": [(-1) ** i * (1 + i % 100 / 128) for i in range(5000)],
          "subnormal beside": [1.25, 2.0 ** -130, 2.0 ** -131, 3 * 2.0 ** -254, 2.0 ** -260]}


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("name", list(VALUES))
def test_largest_values(name, dtype):
    """The factor and the product round to 2^-24 each, the result to its type; its subnormals twice."""
    th = torch()
    x = (th.tensor(VALUES[name], dtype=th.float64) * TOP).to(getattr(th, dtype)).cuda()
    assert x.isfinite().all()
    wide = x.double()
    norm = math.sqrt(math.fsum((wide * wide).tolist()))
    for limit in (1.0, 1.2, 5.0, 1e-30, 0.6 * TOP, 0.999999 * TOP, 1.1 * TOP, 1.99 * TOP):
        say(f"clip_grad_norm {name} {dtype} {limit}")
        out = th.empty_like(x)
        got = og.clip_grad_norm([x], limit, out=[out])
        limit = float(th.tensor(limit))  # (the call takes fp32)
        assert float(got) == float(th.tensor(norm, dtype=th.float64).float())
        want = wide * min(1.0, limit / (norm + 1e-6))
        # (the call's eps is fp32, too: far below any of these norms)
        step = 2.0 ** -23 * 1.01 + th.finfo(x.dtype).eps / 2
        tiny = th.finfo(x.dtype).smallest_normal * th.finfo(x.dtype).eps
        assert ((out.double() - want).abs() <= want.abs() * step * 1.01 + tiny).all(), limit
        mine = x.clone()
        assert og.clip_grad_norm([mine], limit) == got and th.equal(mine, out)
        assert th.equal(og.grad_norm([x]), got)


def test_a_factor_of_one_keeps_every_bit():
    th = torch()
    x = (th.arange(-4000, 4000).cuda() * 2.0 ** -149).float()
    x[0], x[1] = 1.9 * TOP, -1.9 * TOP
    out = th.empty_like(x)
    og.clip_grad_norm([x[2:]], 1.0, out=[out[2:]])
    assert th.equal(out[2:].view(th.int32), x[2:].view(th.int32))
    og.clip_grad_norm([x[:1]], 1.95 * TOP, eps=0.0, out=[out[:1]])
    assert th.equal(out[:1], x[:1])


def test_infinite_elements_beside_large_ones():
    th = torch()
    x = th.tensor([1.9 * TOP, float("inf"), 1.0, -1.9 * TOP], device="cuda")
    assert og.clip_grad_norm([x], 1.0) == float("inf")
    assert x[1].isnan() and (x[[0, 2, 3]] == 0).all()
