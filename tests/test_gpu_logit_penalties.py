"""og_logit_penalties against 64 bits: every step alone and together, histories from none to
long, prompts, repeated and foreign tokens, masks, strides, in place, and what is not written."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu
STEPS = ("repetition", "frequency", "presence", "bias", "mask")


def make(n, v, t, dtype, steps, seed=0, shared=False):
    th = torch()
    gen = th.Generator().manual_seed(seed + 7 * n + v + t)
    c = dict(logits=(3 * th.randn((n, v), generator=gen)).to(getattr(th, dtype)))
    c["tokens"] = th.randint(-2, min(v, 40) + 2, (n, t), generator=gen)
    c["tokens"][:, ::3] = th.randint(0, v, c["tokens"][:, ::3].shape, generator=gen)
    c["lengths"] = th.randint(0, t + 1, (n,), generator=gen)
    c["prompt_lengths"] = (c["lengths"] * th.rand(n, generator=gen)).long()
    c["repetition"] = 0.7 + th.rand(n, generator=gen)
    c["frequency"] = th.rand(n, generator=gen) - 0.2
    c["presence"] = th.rand(n, generator=gen) * 2 - 0.5
    rows, words = 1 if shared else n, (v + 31) // 32
    c["bias"] = th.randn((rows, v), generator=gen)
    c["mask"] = th.randint(-2 ** 31, 2 ** 31, (rows, words), generator=gen).int()
    for s in STEPS:
        if s not in steps:
            c[s] = None
    return {k: None if x is None else x.cuda() for k, x in c.items()}


def check(c, got, **over):
    c = {**c, **over}
    want, bound = ref.logit_penalties(c["logits"], c["tokens"], c["lengths"], c["prompt_lengths"], c["repetition"],
                                      c["frequency"], c["presence"], c["bias"], c["mask"])
    got = got.double().cpu()
    fine = want.isfinite()
    assert ((got - want).abs()[fine] <= bound[fine]).all()
    assert torch().equal(got[~fine].nan_to_num(nan=7.0), want[~fine].nan_to_num(nan=7.0))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("n,v,t", [(1, 1, 1), (1, 4, 1), (3, 31, 5), (2, 33, 0), (5, 1000, 64), (1, 5003, 300),
                                   (4, 4096, 1023), (70, 1023, 17), (2, 40000, 2000)])
def test_all_steps(n, v, t, dtype):
    say(f"logit_penalties {n}x{v} t {t} {dtype}")
    c = make(n, v, t, dtype, STEPS)
    check(c, og.logit_penalties(**c))


@pytest.mark.parametrize("steps", [(s,) for s in STEPS] + [(), ("repetition", "presence"), ("frequency", "mask")])
@pytest.mark.parametrize("v", [2048, 2047])
def test_steps_alone(steps, v):
    say(f"logit_penalties steps {steps} {v}")
    c = make(3, v, 100, "float32", steps, seed=1)
    check(c, og.logit_penalties(**c))


@pytest.mark.parametrize("v", [1536, 1537])
def test_shared_rows_lengths_left_out(v):
    th = torch()
    c = make(6, v, 50, "bfloat16", STEPS, seed=2, shared=True)
    c["lengths"] = c["prompt_lengths"] = None
    check(c, og.logit_penalties(**c))
    check(c, og.logit_penalties(**{**c, "bias": c["bias"][0], "mask": c["mask"][0]}))
    # lengths outside the buffer count as its ends
    far = th.tensor([-5, 10 ** 12, 3, 50, 51, 0], device="cuda")
    early = th.tensor([-3, 20, 10 ** 12, 49, 0, 7], device="cuda")
    got = og.logit_penalties(**{**c, "lengths": far, "prompt_lengths": early})
    check(c, got, lengths=far, prompt_lengths=early)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("steps", [STEPS, ("repetition", "frequency", "presence"), ("bias",), ("mask",)])
@pytest.mark.parametrize("offset,width", [(0, 1064), (3, 1061), (8, 1024)])
def test_strides_and_in_place(steps, offset, width, dtype):
    """Rows inside wider tensors: nothing beside them is written, in place or not."""
    th = torch()
    n = 5
    c = make(n, width, 60, dtype, steps, seed=offset)
    wide = th.full((n, 1072), 7.0, dtype=c["logits"].dtype, device="cuda")
    wide[:, offset:offset + width] = c["logits"]
    view = wide[:, offset:offset + width]
    out = th.full((n, 1100), 9.0, dtype=wide.dtype, device="cuda")
    tokens = th.cat([c["tokens"], th.full((n, 9), 5, device="cuda")], 1)[:, :60]
    given = {**c, "logits": view, "tokens": tokens}
    og.logit_penalties(**given, out=out[:, 4:4 + width])
    check(c, out[:, 4:4 + width])
    assert (out[:, :4] == 9).all() and (out[:, 4 + width:] == 9).all()
    assert th.equal(view, c["logits"])
    assert og.logit_penalties(**given, out=view) is view
    assert th.equal(view, out[:, 4:4 + width])
    assert (wide[:, :offset] == 7).all() and (wide[:, offset + width:] == 7).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("v", [1024, 1021])
def test_special_values(v, dtype):
    """Rows whose mask leaves nothing; infinities, NaN and lowest values in masked and penalised
    places; tokens at the ends of the vocabulary and of their type."""
    th = torch()
    c = make(4, v, 12, dtype, STEPS, seed=5)
    z, inf = c["logits"], float("inf")
    z[:, 0], z[:, 1], z[:, 2], z[:, 3] = inf, -inf, float("nan"), th.finfo(z.dtype).min
    z[:, 4] = th.finfo(z.dtype).max
    c["tokens"][:, :8] = th.tensor([0, 1, 2, 3, v - 1, v, -2 ** 63, 2 ** 63 - 1], device="cuda")
    c["lengths"].fill_(12)
    c["prompt_lengths"][:2] = 0
    c["bias"].fill_(0.5)
    c["mask"][0] = 0
    c["mask"][1] = -1
    c["mask"][2] = 0x55555555
    got = og.logit_penalties(**c)
    check(c, got)
    assert (got[0] == -inf).all()
    assert not got[1].isneginf()[4:].any()
    # a bias of the lowest value
    c["bias"][3] = th.finfo(th.float32).min
    c["bias"][3, 4] = 0
    check(c, og.logit_penalties(**c))


def test_repeated_tokens_count_each_time():
    th = torch()
    v, t = 3000, 20000
    logits = th.zeros((2, v), device="cuda")
    tokens = th.full((2, t), 2999, device="cuda")
    tokens[1, ::2] = 5
    f, p = th.tensor([0.5, 0.25], device="cuda"), th.tensor([1.0, 2.0], device="cuda")
    got = og.logit_penalties(logits, tokens, prompt_lengths=th.tensor([1000, 0], device="cuda"), frequency=f,
                             presence=p)
    assert got[0, 2999] == -0.5 * 19000 - 1 and got[1, 2999] == got[1, 5] == -0.25 * 10000 - 2
    got[:, 2999] = got[:, 5] = 0
    assert (got == 0).all()


def test_empty():
    th = torch()
    e = th.empty((0, 7), device="cuda")
    assert og.logit_penalties(e).shape == (0, 7)
    assert og.logit_penalties(th.empty((3, 0), device="cuda")).shape == (3, 0)
    c = make(3, 70, 0, "float32", ("repetition", "presence"))
    assert th.equal(og.logit_penalties(**c), c["logits"])


def test_refused_by_the_binding():
    th = torch()
    c = make(3, 100, 8, "float32", STEPS)
    bad = [dict(tokens=None), dict(tokens=c["tokens"].int()), dict(tokens=c["tokens"][:2]),
           dict(lengths=c["lengths"].int()), dict(lengths=c["lengths"][:2]), dict(repetition=c["repetition"].double()),
           dict(bias=c["bias"][:, :99]), dict(bias=c["bias"][:2]), dict(bias=c["bias"].half()),
           dict(mask=c["mask"].long()), dict(mask=c["mask"][:, :3]), dict(logits=c["logits"].double()),
           dict(out=c["logits"].half()), dict(out=c["logits"][:2]), dict(bias=c["bias"].cpu()),
           dict(tokens=c["tokens"].t().contiguous().t()), dict(logits=c["logits"].t().contiguous().t())]
    for kw in bad:
        with pytest.raises(ValueError):
            og.logit_penalties(**{**c, **kw})
    shared = {**c, "bias": c["bias"][:1].expand(3, 100)}
    assert th.equal(og.logit_penalties(**shared), og.logit_penalties(**{**c, "bias": c["bias"][:1]}))


def test_more_rows_than_a_launch_has():
    th = torch()
    n, v = 70000, 5
    c = make(n, v, 3, "float32", STEPS, seed=9)
    got = og.logit_penalties(**c)
    for rows in (slice(0, 40), slice(65500, 65570), slice(n - 40, n)):
        part = {k: x[rows] for k, x in c.items()}
        check(part, got[rows])


@pytest.mark.parametrize("width", [1032, 1028, 1027])
def test_in_place_leaves_other_logits_alone(width):
    """Without bias and mask only the row's tokens are written: any bits of the others stay, of a
    NaN too."""
    th = torch()
    z = th.full((2, 1032), 0x7FA12345, dtype=th.int32, device="cuda").view(th.float32)
    view = z[:, :width]
    tokens = th.tensor([[3, width - 1, 3], [700, 0, -1]], device="cuda")
    for i in range(2):
        view[i, tokens[i][tokens[i] >= 0]] = 2.0
    before = z.view(th.int32).clone()
    og.logit_penalties(view, tokens, frequency=th.ones(2, device="cuda"), out=view)
    changed = (z.view(th.int32) != before).nonzero().tolist()
    assert changed == [[0, 3], [0, width - 1], [1, 0], [1, 700]]
    assert view[0, 3] == 0 and view[0, width - 1] == 1 and view[1, 0] == view[1, 700] == 1
