"""The epilogue product, the clipping and the logit penalties with the operators they stand beside,
as they are used: two layers and a head trained (products, cross entropy, gradients, clipping,
orthogonalised update), the head held in 4 bits, its logits penalised; on other streams, captured
and replayed, with kept workspaces, on tensors whose memory other work has used."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch
from test_gpu_lm_run import quantise

pytestmark = pytest.mark.gpu


def inside(got, want, bound):
    assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_train_and_answer(dtype):
    th = torch()
    kind = getattr(th, dtype)
    gen = th.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: th.randn(s, generator=gen, device="cuda")  # noqa: E731
    n, v, d, h = 150, 512, 128, 320
    x, target = rnd(n, d).to(kind), th.randint(0, v, (n,), generator=gen, device="cuda")
    target[::9] = -100
    dloss = th.full((n,), 1.0 / int((target >= 0).sum()), device="cuda")
    up, down, head = (rnd(h, d) / d ** 0.5).to(kind), (rnd(d, h) / h ** 0.5).to(kind), (0.05 * rnd(v, d)).to(kind)
    b_up, b_down = (0.1 * rnd(h)).to(kind), (0.1 * rnd(d)).to(kind)
    for step in range(3):
        say(f"step {step} {dtype}")
        mid, pre = og.gemm_nt_epi(x, up, bias=b_up, act="gelu", need_pre=True)
        e = ref.gemm_epi(x, up, b_up, "gelu", None)
        inside(mid, e["c"], e["e_c"])
        hidden = og.gemm_nt_epi(mid, down, bias=b_down, residual=x)
        e = ref.gemm_epi(mid, down, b_down, None, x)
        inside(hidden, e["c"], e["e_c"])
        loss, lse = og.linear_cross_entropy(hidden, head, target)
        dhidden, dhead = og.linear_cross_entropy_grad(hidden, head, target, lse, dloss)
        dmid, ddown, db_down = og.gemm_nt_epi_grad(dhidden, mid, down)
        dx, dup, db_up = og.gemm_nt_epi_grad(dmid, x, up, pre=pre, act="gelu")
        e = ref.gemm_epi_grad(dmid, x, up, pre, "gelu")
        for got, name in ((dx, "da"), (dup, "dw"), (db_up, "dbias")):
            inside(got, e[name], e["e_" + name])
        grads = [dhead, ddown, db_down, dup, db_up]
        before = [g.clone() for g in grads]
        norm = og.clip_grad_norm(grads, 0.05)
        want = sum(g.double().square().sum() for g in before).sqrt()
        assert (norm.double() - want).abs() <= 2.0 ** -23 * want and want > 0.05
        for g, was in zip(grads, before):
            y = was.double() * 0.05 / (want + 1e-6)
            tiny = th.finfo(kind).smallest_normal * th.finfo(kind).eps
            inside(g, y, y.abs() * (2.0 ** -22 + 1.01 * ref.half_step(kind)) + tiny)
        for w, g in ((head, dhead), (down, ddown), (up, dup)):
            w.copy_(w.float() - 0.02 * og.newton_schulz(g).float())
    q, s, z = quantise(head, 64)
    logits = og.gemm_nt_q4(hidden[:4], q, s, zeros=z, group=64)
    tokens = th.randint(0, v, (4, 40), generator=gen, device="cuda")
    lengths = th.tensor([0, 7, 40, 33], device="cuda")
    ones = th.ones(4, device="cuda")
    mask = th.full((16,), -1, dtype=th.int32, device="cuda")
    mask[3] = 0
    args = dict(lengths=lengths, repetition=1.3 * ones, frequency=0.2 * ones, presence=0.4 * ones, mask=mask)
    got = og.logit_penalties(logits, tokens, **args)
    want, bound = ref.logit_penalties(logits, tokens, lengths, None, 1.3 * ones, 0.2 * ones, 0.4 * ones, None, mask)
    fine = want.isfinite()
    assert ((got.double().cpu() - want).abs()[fine] <= bound[fine]).all()
    assert got[:, 96:128].isneginf().all() and got.isfinite().sum() == 4 * (v - 32)
    assert og.logit_penalties(logits, tokens, **args, out=logits) is logits and th.equal(logits, got)


def state(seed):
    th = torch()
    gen = th.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: th.randn(s, generator=gen, device="cuda")  # noqa: E731
    c = {}
    # few rows, a product in parts, whole tiles, a copy of odd rows
    for name, m, n, k in (("few", 3, 300, 200), ("parts", 200, 192, 2048), ("tiles", 500, 384, 256), ("odd", 130, 77, 301)):
        for kind in ("float32", "bfloat16"):
            to = getattr(th, kind)
            c[name + kind] = dict(a=rnd(m, k).to(to), w=(rnd(n, k) / k ** 0.5).to(to), bias=rnd(n).to(to),
                                  residual=rnd(m, n).to(to), dc=rnd(m, n).to(to))
    c["logits"] = rnd(5, 3000)
    c["tokens"] = th.randint(0, 3000, (5, 500), generator=gen, device="cuda")
    c["lengths"] = th.randint(0, 501, (5,), generator=gen, device="cuda")
    c["f"] = 1 + th.rand(5, generator=gen, device="cuda")
    c["bias"] = rnd(3000)
    return c


def run(c):
    outs, grads = [], []
    for p in c.values():
        if isinstance(p, dict):
            out, pre = og.gemm_nt_epi(p["a"], p["w"], bias=p["bias"], act="silu", residual=p["residual"], need_pre=True)
            grads += og.gemm_nt_epi_grad(p["dc"], p["a"], p["w"], pre=pre, act="silu")
            outs += [out, pre]
    norm = og.clip_grad_norm(grads, 2.0)
    z = og.logit_penalties(c["logits"], c["tokens"], lengths=c["lengths"], repetition=c["f"], frequency=c["f"],
                           presence=c["f"], bias=c["bias"])
    return outs + grads + [norm, z]


def flat(c):
    return [t for p in c.values() for t in (p.values() if isinstance(p, dict) else (p,))]


def test_streams():
    """Two streams at once, each with its own allocations, against the default stream's results."""
    th = torch()
    cases = [state(i) for i in range(2)]
    want = [run(c) for c in cases]
    streams = [th.cuda.Stream() for _ in cases]
    th.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(4):
        for i, s in enumerate(streams):
            with th.cuda.stream(s):
                got[i].append(run(cases[i]))
    th.cuda.synchronize()
    for g, w in zip(got, want):
        for one in g:
            assert all(th.equal(a, b) for a, b in zip(one, w))


def test_graph_replays_match_eager():
    """Captured once, replayed with new inputs in the same tensors, eager work between; the eager
    calls use other workspaces meanwhile."""
    th = torch()
    held = state(0)
    run(held)
    th.cuda.synchronize()
    side, g = th.cuda.Stream(), th.cuda.CUDAGraph()
    with th.cuda.stream(side):
        with th.cuda.graph(g, stream=side):
            outs = run(held)
    th.cuda.synchronize()
    for rep in range(4):
        fresh = state(10 + rep)
        for to, t in zip(flat(held), flat(fresh)):
            to.copy_(t)
        want = [o.clone() for o in run(fresh)]
        for o in outs:
            o.fill_(float("nan"))
        th.cuda.synchronize()
        say(f"replay {rep}")
        g.replay()
        th.cuda.synchronize()
        assert all(th.equal(a, b) for a, b in zip(outs, want)), rep


def test_two_graphs_replayed_together():
    """Two captured runs on two streams at once: each has its workspaces to itself."""
    th = torch()
    cases = [state(20), state(21)]
    want = [[o.clone() for o in run(c)] for c in cases]
    th.cuda.synchronize()
    graphs = []
    for c in cases:
        side, g = th.cuda.Stream(), th.cuda.CUDAGraph()
        with th.cuda.stream(side):
            with th.cuda.graph(g, stream=side):
                outs = run(c)
        graphs.append((side, g, outs))
    for _ in range(3):
        th.cuda.synchronize()
        for side, g, _ in graphs:
            with th.cuda.stream(side):
                g.replay()
    th.cuda.synchronize()
    for (_, _, outs), w in zip(graphs, want):
        assert all(th.equal(a, b) for a, b in zip(outs, w))


CODES = {"float32": og.F32, "bfloat16": og.BF16, "float16": og.F16}


@pytest.mark.parametrize("dtype", list(CODES))
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 300, 200), (40, 100, 3000), (200, 192, 2048), (500, 384, 256),
                                   (130, 77, 301), (90, 1001, 33), (1300, 70, 70)])
@pytest.mark.parametrize("act", [None, "gelu"])
def test_workspaces_of_the_stated_sizes(m, n, k, act, dtype):
    """What a workspace held before does not enter the results, and nothing beside it is written."""
    th = torch()
    gen = th.Generator().manual_seed(m + n + k)
    kind = getattr(th, dtype)
    a, w, bias, dc = (th.randn(s, generator=gen).to(kind).cuda() for s in ((m, k), (n, k), (n,), (m, n)))
    say(f"gemm_nt_epi workspace {m}x{n}x{k} {dtype} {act}")
    sizes = [og.gemm_nt_epi_workspace(m, n, k, CODES[dtype], grad) for grad in (False, True)]
    want = None
    for byte in (0, 0xFF, 0x7B):
        held = [th.full((s + 8192,), byte, dtype=th.uint8, device="cuda") for s in sizes]
        c, pre = og.gemm_nt_epi(a, w, bias=bias, act=act, need_pre=True, workspace=held[0][4096:4096 + sizes[0]])
        got = (c, pre, *og.gemm_nt_epi_grad(dc, a, w, pre=pre, act=act, workspace=held[1][4096:4096 + sizes[1]]))
        assert all(t.isfinite().all() for t in got)
        for t, s in zip(held, sizes):
            assert (t[:4096] == byte).all() and (t[4096 + s:] == byte).all()
        want = want or got
        assert all(th.equal(x, y) for x, y in zip(got, want)), byte


def test_workspace_refusals():
    th = torch()
    a, w, dc = th.ones((200, 2000), device="cuda"), th.ones((600, 2000), device="cuda"), th.ones((200, 600), device="cuda")
    for grad in (False, True):
        size = og.gemm_nt_epi_workspace(200, 600, 2000, og.F32, grad)
        ws = th.empty(size - 1, dtype=th.uint8, device="cuda")
        with pytest.raises(og.OgError):
            og.gemm_nt_epi_grad(dc, a, w, workspace=ws) if grad else og.gemm_nt_epi(a, w, workspace=ws)
        with pytest.raises(ValueError):
            og.gemm_nt_epi(a, w, workspace=ws.cpu())
