"""The language-model operators together, as they are used: a head is trained
(loss, gradient, orthogonalised update), held in 4 bits and asked for single
tokens; on other streams, captured and replayed, with kept workspaces."""
import pytest

import fp32_blocked_gemm_amd as og
import lm_reference as ref
from gpu_util import say, torch

pytestmark = pytest.mark.gpu


def quantise(w, group):
    """Codes, scales and zero points of w by rounding to the nearest in each group."""
    t = torch()
    n, k = w.shape
    parts = w.float().view(n, k // group, group)
    low, high = parts.amin(2).clamp(max=0), parts.amax(2).clamp(min=0)
    s = ((high - low) / 15).clamp(min=1e-8)
    z = t.round(-low / s).clamp(0, 15)
    q = t.round(parts / s[:, :, None] + z[:, :, None]).clamp(0, 15).to(t.uint8).view(n, k)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s, z.to(t.uint8)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_train_update_quantise_answer(dtype):
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(0)
    n, v, d = 200, 1024, 256
    kind = getattr(t, dtype)
    w = (t.randn((v, d), generator=gen, device="cuda") * 0.02).to(kind)
    x = t.randn((n, d), generator=gen, device="cuda").to(kind)
    target = t.randint(0, v, (n,), generator=gen, device="cuda")
    target[::7] = -100
    dloss = t.full((n,), 1.0 / int((target >= 0).sum()), device="cuda")
    momentum = t.zeros_like(w)
    for step in range(3):
        say(f"step {step} {dtype}")
        loss, lse = og.linear_cross_entropy(x, w, target)
        dx, dw = og.linear_cross_entropy_grad(x, w, target, lse, dloss)
        e = ref.cross_entropy(x, w, target, -100, dloss)
        assert ((loss.double() - e["loss"]).abs() <= e["e_loss"]).all()
        assert ((dw.double() - e["dw"]).abs() <= e["e_dw"]).all()
        assert ((dx.double() - e["dx"]).abs() <= e["e_dx"]).all()
        momentum = 0.9 * momentum + dw
        update = og.newton_schulz(momentum)
        exact, bound = ref.newton_schulz(momentum, 5, (3.4445, -4.7750, 2.0315), 1e-7)
        assert (update.double() - exact).norm() <= bound
        w = (w.float() - 0.02 * update.float()).to(kind)
    q, s, z = quantise(w, 64)
    token = x[3:4]
    logits = og.gemm_nt_q4(token, q, s, zeros=z, group=64)
    exact, bound = ref.q4(token, q, s, z, 64)
    assert ((logits.double() - exact).abs() <= bound).all()
    # scoring against the same weights, written out: the lse of the 4-bit logits
    held = ref.q4_weights(q, s, z, d, 64).float()
    _, lse = og.linear_cross_entropy(token.float(), held, target[3:4])
    e = ref.cross_entropy(token.float(), held, target[3:4], -100, None)
    assert ((lse.double() - e["lse"]).abs() <= e["e_lse"]).all()


def state(seed):
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: t.randn(s, generator=gen, device="cuda")  # noqa: E731
    n, v, d = 90, 700, 128
    target = t.randint(0, v, (n,), generator=gen, device="cuda")
    target[::5] = -100
    q, s, z = quantise(0.02 * rnd(v, d), 32)
    return dict(x=rnd(n, d).bfloat16(), w=(0.05 * rnd(v, d)).bfloat16(), target=target, dloss=rnd(n),
                q=q, s=s, z=z)


def run(c):
    loss, lse = og.linear_cross_entropy(c["x"], c["w"], c["target"])
    dx, dw = og.linear_cross_entropy_grad(c["x"], c["w"], c["target"], lse, c["dloss"])
    x32, w32 = c["x"].float(), c["w"].float()
    loss32, lse32 = og.linear_cross_entropy(x32, w32, c["target"])
    dx32, dw32 = og.linear_cross_entropy_grad(x32, w32, c["target"], lse32, c["dloss"])
    up = og.newton_schulz(dw32)
    up16 = og.newton_schulz(dw)
    y = og.gemm_nt_q4(c["x"][:4], c["q"], c["s"], zeros=c["z"], group=32)
    return loss, lse, dx, dw, loss32, lse32, dx32, dw32, up, up16, y


def test_streams():
    """Two streams at once, each with its own allocations, against the default stream's results."""
    t = torch()
    cases = [state(i) for i in range(2)]
    want = [run(c) for c in cases]
    streams = [t.cuda.Stream() for _ in cases]
    t.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(5):
        for i, s in enumerate(streams):
            with t.cuda.stream(s):
                got[i].append(run(cases[i]))
    t.cuda.synchronize()
    for g, w in zip(got, want):
        for one in g:
            assert all(t.equal(a, b) for a, b in zip(one, w))


def test_graph_replays_match_eager():
    """Captured once, replayed with new inputs in the same tensors, eager work between."""
    t = torch()
    held = state(0)
    run(held)
    t.cuda.synchronize()
    side, g = t.cuda.Stream(), t.cuda.CUDAGraph()
    with t.cuda.stream(side):
        with t.cuda.graph(g, stream=side):
            outs = run(held)
    t.cuda.synchronize()
    for rep in range(4):
        fresh = state(10 + rep)
        for name in held:
            held[name].copy_(fresh[name])
        want = [o.clone() for o in run(fresh)]
        for o in outs:
            o.fill_(float("nan"))
        t.cuda.synchronize()
        say(f"replay {rep}")
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(outs, want)), rep


def test_kept_workspaces():
    """A caller's own workspace of exactly the stated size, used by call after call, its other
    bytes untouched; one that is too small is refused."""
    t = torch()
    c = state(3)
    n, d = c["x"].shape
    v = c["w"].shape[0]
    sizes = [og.linear_cross_entropy_workspace(n, v, d, og.BF16),
             og.linear_cross_entropy_workspace(n, v, d, og.BF16, grad=True),
             og.newton_schulz_workspace(1, v, d, og.BF16)]
    ws = []
    for s in sizes:
        whole = t.full((s + 4096,), 0xA5, dtype=t.uint8, device="cuda")
        ws.append((whole, whole[:s]))
    want = run(c)
    for _ in range(2):
        loss, lse = og.linear_cross_entropy(c["x"], c["w"], c["target"], workspace=ws[0][1])
        dx, dw = og.linear_cross_entropy_grad(c["x"], c["w"], c["target"], lse, c["dloss"], workspace=ws[1][1])
        up = og.newton_schulz(dw, workspace=ws[2][1])
        for a, b in zip((loss, lse, dx, dw, up), (*want[:4], want[9])):
            assert t.equal(a, b)
    for (whole, part), s in zip(ws, sizes):
        assert (whole[s:] == 0xA5).all()
    with pytest.raises(og.OgError):
        og.newton_schulz(dw, workspace=ws[2][1][:-1])
    with pytest.raises(ValueError):
        og.newton_schulz(dw, workspace=ws[2][1].cpu())
