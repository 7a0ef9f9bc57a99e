"""What is timed of the language-model operators around the N x K product.

Three operators, each beside og_gemm_nt_f32 (a right operand whose rows hold
the k weights of one output):

- gemm_nt_q4: C = A W^T with W held in 4 bits and a scale (and a zero point)
  for each group of k;
- linear_cross_entropy and its gradient: the softmax cross entropy of X W^T
  over a large vocabulary, the logits never kept;
- newton_schulz: the orthogonalised update of a matrix gradient by a chain of
  products (X <- a X + (b A + c A A) X with A = X X^T).

`run` computes them in elementary torch operations in 32 bits, or, where
`own` is true, by this package's calls; `exact` computes them in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
IGNORE = -100


def listed():
    return [
        # one token through a 4096-wide projection: the smallest call of a decoder, latency decides
        {"name": "q4 token 4096x4096 bf16", "op": "q4", "m": 1, "n": 4096, "k": 4096, "group": 128,
         "type": "bf16", "scales": "bf16", "zeros": False},
        # one token through the up projection in 32 bits, fine groups with zero points
        {"name": "q4 token 11008x4096 f32 zeros", "op": "q4", "m": 1, "n": 11008, "k": 4096, "group": 32,
         "type": "f32", "scales": "f32", "zeros": True},
        # sixteen sequences decoded together
        {"name": "q4 batch 16 4096x11008 f16", "op": "q4", "m": 16, "n": 4096, "k": 11008, "group": 64,
         "type": "f16", "scales": "f16", "zeros": True},
        # an odd layer: ragged n, a last group that is not full
        {"name": "q4 ragged 7x1531x1000 bf16", "op": "q4", "m": 7, "n": 1531, "k": 1000, "group": 128,
         "type": "bf16", "scales": "f32", "zeros": False},
        # the log-probability of one token (scoring while decoding): the weights are streamed once
        {"name": "ce score 1x32768x4096 bf16", "op": "ce", "n": 1, "v": 32768, "d": 4096, "type": "bf16",
         "train": False, "ignored": 0.0},
        # scoring a prompt against a vocabulary of odd length
        {"name": "ce score 777x50021x768 f32", "op": "ce", "n": 777, "v": 50021, "d": 768, "type": "f32",
         "train": False, "ignored": 0.1},
        # a training step of a small model, padded batch, 32 bits
        {"name": "ce train 1000x8191x384 f32", "op": "ce", "n": 1000, "v": 8191, "d": 384, "type": "f32",
         "train": True, "ignored": 0.3},
        # a training step of a large one
        {"name": "ce train 4096x32768x4096 bf16", "op": "ce", "n": 4096, "v": 32768, "d": 4096, "type": "bf16",
         "train": True, "ignored": 0.05},
        # a small projection: fifteen dependent products, latency decides
        {"name": "ns 128x512 f32", "op": "ns", "count": 1, "m": 128, "n": 512, "type": "f32"},
        # odd sizes, more rows than columns
        {"name": "ns 1531x777 bf16", "op": "ns", "count": 1, "m": 1531, "n": 777, "type": "bf16"},
        # the twelve attention outputs of a 768-wide encoder at once
        {"name": "ns 12 of 768x768 f32", "op": "ns", "count": 12, "m": 768, "n": 768, "type": "f32"},
        # a feed-forward matrix of a 4096-wide model
        {"name": "ns 4096x11008 bf16", "op": "ns", "count": 1, "m": 4096, "n": 11008, "type": "bf16"},
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("q4", "ce", "ns"))
    if op == "q4":
        return {"op": "q4", "m": _log(rng, 1, 64), "n": _log(rng, 500, 12000), "k": _log(rng, 500, 12000),
                "group": rng.choice((32, 64, 128)), "type": rng.choice(("f32", "bf16", "f16")),
                "scales": rng.choice(("f32", "bf16", "f16")), "zeros": rng.random() < 0.5}
    if op == "ce":
        return {"op": "ce", "n": _log(rng, 1, 4096), "v": _log(rng, 1000, 32768),
                "d": 8 * _log(rng, 16, 512) - (rng.randrange(8) if rng.random() < 0.3 else 0),
                "type": rng.choice(("f32", "bf16")), "train": rng.random() < 0.6,
                "ignored": rng.choice((0.0, 0.1, 0.5))}
    return {"op": "ns", "count": rng.choice((1, 1, 2, 5)), "m": _log(rng, 50, 4096), "n": _log(rng, 50, 2048),
            "type": rng.choice(("f32", "bf16"))}


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _inputs(case, seed):
    """The tensors of a case, on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = TYPES[case["type"]]
    if case["op"] == "q4":
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        groups = -(-k // group)
        a = _normal((m, k), gen).to(t)
        w = torch.zeros((n, groups * group), device="cuda")
        w[:, :k] = _normal((n, k), gen, 0.02)
        w = w.view(n, groups, group)
        # round to nearest in each group: symmetric about the code 8, or from the group's lowest to its highest value
        if case["zeros"]:
            low, high = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
            scales = ((high - low) / 15).to(TYPES[case["scales"]])
            zeros = torch.round(-low / scales.float()).clamp(0, 15)
        else:
            scales = (w.abs().amax(2) / 7).to(TYPES[case["scales"]])
            zeros = torch.full((n, groups), 8.0, device="cuda")
        codes = torch.round(w / scales.float()[:, :, None] + zeros[:, :, None]).clamp(0, 15).to(torch.uint8)
        codes = codes.view(n, -1)[:, : k + (k & 1)]
        return {"a": a, "q": (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), "scales": scales.contiguous(),
                "zeros": zeros.to(torch.uint8).contiguous() if case["zeros"] else None}
    if case["op"] == "ce":
        n, v, d = case["n"], case["v"], case["d"]
        w = _normal((v, d), gen, 0.02)
        target = torch.randint(0, v, (n,), generator=gen, device="cuda")
        # hidden states that know something of their token: its logit stands out by 0 to 10
        lift = 10 * torch.rand((n, 1), generator=gen, device="cuda") / (0.0004 * d)
        x = _normal((n, d), gen) + lift * w[target]
        drop = torch.rand((n,), generator=gen, device="cuda") < case["ignored"]
        target = torch.where(drop, torch.full_like(target, IGNORE), target)
        # the mean over the tokens that count, as a training step weighs them
        dloss = torch.ones((n,), device="cuda") / (~drop).sum().clamp(min=1)
        return {"x": x.to(t), "w": w.to(t), "target": target, "dloss": dloss}
    c, m, n = case["count"], case["m"], case["n"]
    rank = max(1, min(m, n) // 8)
    # a gradient: a few strong directions over a noise floor
    g = (_normal((c, m, rank), gen) @ _normal((c, rank, n), gen)) / math.sqrt(rank) + 0.3 * _normal((c, m, n), gen)
    return {"g": (0.01 * g).to(t).squeeze(0) if c == 1 else (0.01 * g).to(t)}


def prepare(case, seed):
    return {"case": case, **_inputs(case, seed)}


def _dequantised(q, scales, zeros, k, group, dtype):
    codes = torch.stack((q & 15, q >> 4), 2).view(q.shape[0], -1)[:, :k].to(dtype)
    at = torch.arange(k, device=q.device) // group
    zero = zeros.to(dtype)[:, at] if zeros is not None else 8
    return (codes - zero) * scales.to(dtype)[:, at]


def _q4(s):
    c = s["case"]
    if own:
        import fp32_blocked_gemm_amd as og
        return og.gemm_nt_q4(s["a"], s["q"], s["scales"], zeros=s["zeros"], group=c["group"])
    w = _dequantised(s["q"], s["scales"], s["zeros"], c["k"], c["group"], torch.float32)
    return (s["a"].float() @ w.t()).to(s["a"].dtype)


def _ce(s):
    x, w, target, dloss, train = s["x"], s["w"], s["target"], s["dloss"], s["case"]["train"]
    if own:
        import fp32_blocked_gemm_amd as og
        loss, lse = og.linear_cross_entropy(x, w, target, ignore_index=IGNORE)
        if not train:
            return {"loss": loss, "lse": lse}
        dx, dw = og.linear_cross_entropy_grad(x, w, target, lse, dloss, ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    counts = target != IGNORE
    at = torch.where(counts, target, torch.zeros_like(target))[:, None]
    x32, w32 = x.float(), w.float()
    z = x32 @ w32.t()
    top = z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    zero = torch.zeros_like(lse)
    loss = torch.where(counts, lse - z.gather(1, at)[:, 0], zero)
    if not train:
        return {"loss": loss, "lse": torch.where(counts, lse, zero)}
    g = torch.exp(z - lse[:, None])
    g.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    g = torch.where(counts[:, None], g * dloss[:, None], zero[:, None])
    return {"loss": loss, "lse": torch.where(counts, lse, zero), "dx": (g @ w32).to(x.dtype),
            "dw": (g.t() @ x32).to(w.dtype)}


def _step(x):
    a = x @ x.transpose(-2, -1)
    return COEFFS[0] * x + (COEFFS[1] * a + COEFFS[2] * (a @ a)) @ x


def _chain(g, dtype):
    """Five steps from g over its norm, the shorter side first."""
    x = g.to(dtype)
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    tall = g.shape[-2] > g.shape[-1]
    x = x.transpose(-2, -1).contiguous() if tall else x
    x = _step(_step(_step(_step(_step(x)))))
    return x.transpose(-2, -1).contiguous() if tall else x


def _ns(s):
    if own:
        import fp32_blocked_gemm_amd as og
        return og.newton_schulz(s["g"], steps=5, coeffs=COEFFS, eps=EPS)
    return _chain(s["g"], torch.float32).to(s["g"].dtype)


def run(state):
    return {"q4": _q4, "ce": _ce, "ns": _ns}[state["case"]["op"]](state)


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    b = size[case["type"]]
    if case["op"] == "q4":
        m, n, k = case["m"], case["n"], case["k"]
        groups = -(-k // case["group"])
        held = n * ((k + 1) // 2) + n * groups * (size[case["scales"]] + (1 if case["zeros"] else 0))
        return {"bytes": held + b * m * (k + n), "flops": 2 * m * n * k}
    if case["op"] == "ce":
        n, v, d = case["n"], case["v"], case["d"]
        read, out = b * (n * d + v * d) + 8 * n, 8 * n
        if not case["train"]:
            return {"bytes": read + out, "flops": 2 * n * v * d}
        # the logits, then the two products of their gradient
        return {"bytes": read + out + 4 * n + b * (n * d + v * d), "flops": 6 * n * v * d}
    c, r, k = case["count"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # X X^T and A A are symmetric: half of each is enough
    return {"bytes": 2 * b * c * r * k, "flops": 5 * c * (r * r * k + r * r * r + 2 * r * r * k)}


def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    if case["op"] == "q4":
        k = case["k"]
        w = torch.empty((case["n"], 2 * s["q"].shape[1]), dtype=f, device="cuda")
        w[:, 0::2], w[:, 1::2] = (s["q"] % 16).to(f), (s["q"] // 16).to(f)
        spread = lambda t: t.to(f).repeat_interleave(case["group"], 1)[:, :k]  # noqa: E731
        w = (w[:, :k] - (spread(s["zeros"]) if case["zeros"] else 8.0)) * spread(s["scales"])
        return torch.matmul(w, s["a"].to(f).t()).t().contiguous()
    if case["op"] == "ce":
        x, w = s["x"].to(f), s["w"].to(f)
        keep = (s["target"] >= 0).nonzero()[:, 0]
        rows, t = x[keep], s["target"][keep]
        logp = torch.log_softmax(torch.matmul(rows, w.t()), 1)
        at = torch.arange(len(keep), device="cuda")
        loss, lse = torch.zeros(len(x), dtype=f, device="cuda"), torch.zeros(len(x), dtype=f, device="cuda")
        loss[keep] = -logp[at, t]
        lse[keep] = (rows * w[t]).sum(1) - logp[at, t]
        if not case["train"]:
            return {"loss": loss, "lse": lse}
        p = logp.exp_()
        p[at, t] -= 1
        p *= s["dloss"].to(f)[keep][:, None]
        dx = torch.zeros_like(x)
        dx[keep] = torch.matmul(p, w)
        return {"loss": loss, "lse": lse, "dx": dx, "dw": torch.matmul(p.t(), rows)}
    # the same polynomial from the other side: X <- X (a I + b S + c S S), S = X^T X, where that is the smaller matrix
    a, b, c = COEFFS
    out = []
    for g in s["g"].to(f).reshape(-1, case["m"], case["n"]):
        x = g / (torch.linalg.vector_norm(g) + EPS)
        eye = torch.eye(min(x.shape), dtype=f, device="cuda")
        for _ in range(5):
            if x.shape[0] >= x.shape[1]:
                gram = x.t() @ x
                x = x @ (a * eye + b * gram + c * gram @ gram)
            else:
                gram = x @ x.t()
                x = (a * eye + b * gram + c * gram @ gram) @ x
        out.append(x)
    return torch.stack(out).reshape(s["g"].shape)
