"""og_logit_penalties in place without bias and mask: a logit that no penalty changes keeps its bits, next to
others that are changed, in whole vectors of eight, single logits and the last, partial vector."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
# a signalling NaN, which a conversion to fp32 and back would make quiet
BITS = {"float32": (0x7FA12345, "int32"), "bfloat16": (0x7F81, "int16"), "float16": (0x7C01, "int16")}


@pytest.mark.parametrize("dtype", list(BITS))
@pytest.mark.parametrize("width", [1032, 1027])
@pytest.mark.parametrize("steps", [("repetition",), ("frequency",), ("presence",), ("frequency", "presence"),
                                   ("repetition", "frequency", "presence")])
def test_only_penalised_logits_change(steps, width, dtype):
    th = torch()
    bits, whole = BITS[dtype]
    raw = th.full((3, 1040), bits, dtype=getattr(th, whole), device="cuda")
    z = raw.view(getattr(th, dtype))[:, :width]
    tokens = th.tensor([[3, width - 1, 9, 3], [700, 0, -1, 9], [5, 6, 7, 8]], device="cuda")
    prompt = th.tensor([2, 1, 4], device="cuda")
    # (row 0: 3 and the last are in its prompt, 9 and 3 are generated; row 2 has a prompt only)
    generated = [{9, 3}, {0, 9}, set()]
    seen = [{3, 9, width - 1}, {700, 0, 9}, {5, 6, 7, 8}]
    changed = seen if "repetition" in steps else generated
    for i in range(3):
        for j in changed[i]:
            z[i, j] = 2.0
    was, before = raw.clone(), z.clone()
    given = {s: th.full((3,), 1.25, device="cuda") for s in steps}
    say(f"logit_penalties in place {steps} {width} {dtype}")
    og.logit_penalties(z, tokens, prompt_lengths=prompt, out=z, **given)
    places = {(i, j) for i in range(3) for j in changed[i]}
    assert {tuple(p) for p in (raw != was).nonzero().tolist()} == places
    want, bound = ref.logit_penalties(before, tokens, None, prompt, *(given.get(s) for s in (
        "repetition", "frequency", "presence")), None, None)
    for i, j in places:
        assert abs(float(z[i, j]) - float(want[i, j])) <= float(bound[i, j])


@pytest.mark.parametrize("dtype", list(BITS))
def test_in_place_as_out_of_place(dtype):
    th = torch()
    gen = th.Generator().manual_seed(3)
    z = (3 * th.randn((6, 40000), generator=gen)).to(getattr(th, dtype)).cuda()
    tokens = th.randint(0, 40000, (6, 9000), generator=gen).cuda()
    prompt = th.randint(0, 9000, (6,), generator=gen).cuda()
    f = (1 + th.rand(6, generator=gen)).cuda()
    args = dict(prompt_lengths=prompt, repetition=f, frequency=f, presence=f)
    want = og.logit_penalties(z, tokens, **args)
    assert og.logit_penalties(z, tokens, out=z, **args) is z and th.equal(z, want)
