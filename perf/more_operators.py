"""What is timed of the operators around training a layer and answering with its logits.

Three operators, beside og_gemm_nt_f32 and the operators that train, update
and answer with its N x K weights:

- gemm_nt_epi: C = act(A W^T + bias) + residual, and its gradient: the layers
  before a language model's head;
- clip_grad_norm: the norm over all gradients of a model, and the gradients
  scaled down to a largest norm, before the update;
- logit_penalties: penalties for the tokens a sequence already holds, biases
  and a mask of allowed tokens on the logits of each row, before a token is
  drawn.

`run` computes them in elementary torch operations in 32 bits, or, where
`own` is true, by this package's calls; `exact` computes them in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
MAX_NORM = 1.0
EPS = 1e-6


def listed():
    return [
        # one token through a 4096-wide model's up projection: latency and the weights' bytes
        {"name": "epi token 1x11008x4096 bf16 silu", "op": "epi", "m": 1, "n": 11008, "k": 4096, "type": "bf16",
         "act": "silu", "bias": False, "residual": False, "train": False},
        # sixteen sequences decoded together through the down projection, back onto the residual stream
        {"name": "epi batch 16x4096x11008 f16 residual", "op": "epi", "m": 16, "n": 4096, "k": 11008, "type": "f16",
         "act": "none", "bias": True, "residual": True, "train": False},
        # odd sizes in 32 bits
        {"name": "epi 777x1531x1000 f32 gelu", "op": "epi", "m": 777, "n": 1531, "k": 1000, "type": "f32",
         "act": "gelu", "bias": True, "residual": False, "train": False},
        # a prompt in 32 bits
        {"name": "epi prompt 512x11008x4096 f32 relu", "op": "epi", "m": 512, "n": 11008, "k": 4096, "type": "f32",
         "act": "relu", "bias": True, "residual": False, "train": False},
        # a training step of a 384-wide encoder's feed-forward layer, forward and gradients
        {"name": "epi train 4096x1536x384 f32 gelu", "op": "epi", "m": 4096, "n": 1536, "k": 384, "type": "f32",
         "act": "gelu", "bias": True, "residual": False, "train": True},
        # a training step of a 4096-wide model's up projection
        {"name": "epi train 4096x11008x4096 bf16 silu", "op": "epi", "m": 4096, "n": 11008, "k": 4096, "type": "bf16",
         "act": "silu", "bias": True, "residual": False, "train": True},
        # the adapters or the head alone: a few small gradients, latency decides
        {"name": "clip 1 layer of 128 f32", "op": "clip", "layers": 1, "width": 128, "inner": 512, "vocab": 0,
         "type": "f32", "norm": 3.0},
        # every gradient of a 384-wide encoder with its embedding of odd length
        {"name": "clip 6 layers of 384 f32", "op": "clip", "layers": 6, "width": 384, "inner": 1536, "vocab": 30001,
         "type": "f32", "norm": 20.0},
        # two layers and the head of a 4096-wide model, weights in 16 bits and norms in 32
        {"name": "clip 2 layers of 4096 bf16", "op": "clip", "layers": 2, "width": 4096, "inner": 11008,
         "vocab": 32768, "type": "bf16", "norm": 7.0},
        # one sequence: a short text, no grammar
        {"name": "penalties 1x32768 f32", "op": "penalties", "rows": 1, "vocab": 32768, "tokens": 200, "type": "f32",
         "bias": False, "mask": False},
        # a few long sequences against a vocabulary of odd length
        {"name": "penalties 9x50021 f32 long", "op": "penalties", "rows": 9, "vocab": 50021, "tokens": 16384,
         "type": "f32", "bias": True, "mask": False},
        # a full batch under grammars
        {"name": "penalties 64x131072 bf16 mask", "op": "penalties", "rows": 64, "vocab": 131072, "tokens": 2000,
         "type": "bf16", "bias": True, "mask": True},
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("epi", "epi", "clip", "penalties"))
    if op == "epi":
        kind = rng.choice(("f32", "bf16", "f16"))
        step = rng.choice((1, 8))
        n, k = (step * _log(rng, 64 // step, (4096 if kind == "f32" else 11008) // step) for _ in range(2))
        return {"op": "epi", "m": _log(rng, 1, 4096), "n": n, "k": min(k, 4096), "type": kind,
                "act": rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.4, "train": rng.random() < 0.5}
    if op == "clip":
        width = _log(rng, 64, 2048)
        return {"op": "clip", "layers": _log(rng, 1, 6), "width": width, "inner": 4 * width - rng.randrange(3),
                "vocab": rng.choice((0, _log(rng, 1000, 50000))), "type": rng.choice(("f32", "bf16", "f16", "mixed")),
                "norm": rng.choice((0.5, 3.0, 50.0))}
    return {"op": "penalties", "rows": _log(rng, 1, 64), "vocab": _log(rng, 1000, 131072), "tokens": _log(rng, 1, 16384),
            "type": rng.choice(("f32", "bf16", "f16")), "bias": rng.random() < 0.5, "mask": rng.random() < 0.5}


def _normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _uniform(shape, gen, low=0.0, high=1.0):
    return torch.rand(shape, generator=gen, device="cuda") * (high - low) + low


def _shapes(case):
    """(shape, type) of each gradient of a model: four square projections, a gated feed-forward
    layer and two norms for each layer, and the embedding."""
    w, i = case["width"], case["inner"]
    kind = "bf16" if case["type"] == "mixed" else case["type"]
    vector = "f32" if case["type"] in ("mixed", "bf16") else kind
    layer = [((w, w), kind)] * 4 + [((i, w), kind)] * 2 + [((w, i), kind)] + [((w,), vector)] * 2
    return layer * case["layers"] + ([((case["vocab"], w), kind)] if case["vocab"] else [])


def _inputs(case, seed):
    """The tensors of a case, on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "epi":
        m, n, k, t = case["m"], case["n"], case["k"], TYPES[case["type"]]
        # the gradient of a mean over the tokens, some of which are padding
        drop = _uniform((m, 1), gen) < 0.05
        dc = torch.where(drop, torch.zeros((), device="cuda"), _normal((m, n), gen, 0.02))
        return {"a": _normal((m, k), gen).to(t), "w": _normal((n, k), gen, k ** -0.5).to(t),
                "bias": _normal((n,), gen, 0.2).to(t) if case["bias"] else None,
                "residual": _normal((m, n), gen).to(t) if case["residual"] else None,
                "dc": dc.to(t) if case["train"] else None}
    if case["op"] == "clip":
        shapes = _shapes(case)
        # layers' gradients differ in size; all of them together have about the case's norm
        sizes = [math.prod(s) for s, _ in shapes]
        std = [0.5 + ((7 * i) % 10) / 10 for i in range(len(shapes))]
        unit = case["norm"] / math.sqrt(sum(n * s * s for n, s in zip(sizes, std)))
        grads = [_normal(shape, gen, unit * s).to(TYPES[kind]) for (shape, kind), s in zip(shapes, std)]
        return {"grads": grads, "out": [torch.empty_like(g) for g in grads]}
    r, v, most, t = case["rows"], case["vocab"], case["tokens"], TYPES[case["type"]]
    lengths = torch.randint((most + 1) // 2, most + 1, (r,), generator=gen, device="cuda")
    # text repeats its common tokens: density falls off with the token's place
    tokens = (v * _uniform((r, most), gen) ** 4).long().clamp(max=v - 1)
    tokens = (tokens * 7919 + 13) % v
    tokens = torch.where(torch.arange(most, device="cuda") < lengths[:, None], tokens, torch.full_like(tokens, -1))
    bias = mask = None
    if case["bias"]:
        chosen = _uniform((v,), gen)
        bias = torch.where(chosen < 0.01, _normal((v,), gen, 5.0), torch.zeros((), device="cuda"))
    if case["mask"]:
        # a grammar allows few tokens in some rows and nearly all of them in others
        share = _uniform((r, 1), gen) ** 3
        words = (v + 31) // 32
        allowed = (_uniform((r, words * 32), gen) < share).view(r, words, 32).long()
        mask = (allowed << torch.arange(32, device="cuda")).sum(2)
        mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).int()
    return {"logits": _normal((r, v), gen, 3.0).to(t), "tokens": tokens, "lengths": lengths,
            "prompt": (lengths * _uniform((r,), gen)).long(), "repetition": _uniform((r,), gen, 1.0, 1.5),
            "frequency": _uniform((r,), gen, 0.0, 0.8), "presence": _uniform((r,), gen, 0.0, 1.5), "bias": bias,
            "mask": mask}


def prepare(case, seed):
    return {"case": case, **_inputs(case, seed)}


def _act(x, act):
    """act(x) and its derivative."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        on = (x > 0).float()
        return x * on, on
    if act == "gelu":
        below = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        return x * below, below + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (x + 0.044715 * x * x * x))
        return x * s, s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x * x)
    s = torch.sigmoid(x)
    return x * s, s * (1 + x * (1 - s))


def _epi(s):
    c, a, w, bias, residual, dc = s["case"], s["a"], s["w"], s["bias"], s["residual"], s["dc"]
    act = None if c["act"] == "none" else c["act"]
    if own:
        import fp32_blocked_gemm_amd as og
        if not c["train"]:
            return og.gemm_nt_epi(a, w, bias=bias, act=act, residual=residual)
        out, pre = og.gemm_nt_epi(a, w, bias=bias, act=act, residual=residual, need_pre=True)
        da, dw, dbias = og.gemm_nt_epi_grad(dc, a, w, pre=pre, act=act, need=(True, True, c["bias"]))
        return {"c": out, "da": da, "dw": dw, **({"dbias": dbias} if c["bias"] else {})}
    t = a.dtype
    a, w = a.float(), w.float()
    x = a @ w.t()
    x = x + bias.float() if c["bias"] else x
    y, slope = _act(x, c["act"])
    out = (y + residual.float() if c["residual"] else y).to(t)
    if not c["train"]:
        return out
    dp = dc.float() * slope
    got = {"c": out, "da": (dp @ w).to(t), "dw": (dp.t() @ a).to(t)}
    return {**got, "dbias": dp.sum(0).to(t)} if c["bias"] else got


def _clip(s):
    grads, out = s["grads"], s["out"]
    if own:
        import fp32_blocked_gemm_amd as og
        return {"norm": og.clip_grad_norm(grads, MAX_NORM, eps=EPS, out=out), "grads": out}
    # (squares summed in 64 bits: a long sum)
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()
    by = (MAX_NORM / (norm + EPS)).clamp(max=1.0).float()
    return {"norm": norm.float(), "grads": [(g.float() * by).to(g.dtype) for g in grads]}


def _penalties(s):
    z, tokens, lengths, prompt, bias, mask = (s[i] for i in ("logits", "tokens", "lengths", "prompt", "bias", "mask"))
    if own:
        import fp32_blocked_gemm_amd as og
        return og.logit_penalties(z, tokens, lengths=lengths, prompt_lengths=prompt, repetition=s["repetition"],
                                  frequency=s["frequency"], presence=s["presence"], bias=bias, mask=mask,
                                  out=torch.empty_like(z))
    rows, v = z.shape
    place = torch.arange(tokens.shape[1], device=z.device)
    held = place < lengths[:, None]
    at = torch.where(held, tokens, torch.zeros_like(tokens))
    seen = torch.zeros((rows, v), device=z.device).scatter_add_(1, at, held.float())
    count = torch.zeros((rows, v), device=z.device).scatter_add_(1, at, (held & (place >= prompt[:, None])).float())
    x, r = z.float(), s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    x = x + bias if bias is not None else x
    if mask is not None:
        bits = (mask[:, :, None] >> torch.arange(32, device=z.device, dtype=torch.int32)) & 1
        x = torch.where(bits.reshape(rows, -1)[:, :v] > 0, x, torch.full((), -math.inf, device=z.device))
    return x.to(z.dtype)


def run(state):
    return {"epi": _epi, "clip": _clip, "penalties": _penalties}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "epi":
        m, n, k = case["m"], case["n"], case["k"]
        values = m * k + n * k + m * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)
        if case["train"]:
            # dC, then dA, dW and dbias
            values += m * n + m * k + n * k + (n if case["bias"] else 0)
        return {"bytes": SIZE[case["type"]] * values, "flops": (6 if case["train"] else 2) * m * n * k}
    if case["op"] == "clip":
        return {"bytes": 2 * sum(SIZE[kind] * math.prod(shape) for shape, kind in _shapes(case)),
                "flops": 3 * sum(math.prod(shape) for shape, _ in _shapes(case))}
    r, v = case["rows"], case["vocab"]
    held = 2 * SIZE[case["type"]] * r * v + 6 * r * case["tokens"] + 28 * r
    return {"bytes": held + (4 * v if case["bias"] else 0) + (r * ((v + 31) // 32) * 4 if case["mask"] else 0),
            "flops": r * v * (1 + case["bias"]) + 6 * r * case["tokens"]}


def _exact_penalties(case, s):
    """A row at a time, by its sorted tokens."""
    rows = []
    for i in range(case["rows"]):
        x = s["logits"][i].double()
        length, prompt = int(s["lengths"][i]), int(s["prompt"][i])
        every = torch.unique(s["tokens"][i, :length])
        x[every] = torch.where(x[every] > 0, x[every] / s["repetition"][i].double(),
                               x[every] * s["repetition"][i].double())
        made, times = torch.unique(s["tokens"][i, prompt:length], return_counts=True)
        x[made] -= s["frequency"][i].double() * times + s["presence"][i].double()
        if s["bias"] is not None:
            x += s["bias"].double()
        if s["mask"] is not None:
            token = torch.arange(case["vocab"], device="cuda")
            x[(s["mask"][i].long()[token // 32] // (1 << (token % 32))) % 2 == 0] = -math.inf
        rows.append(x)
    return torch.stack(rows)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "penalties":
        return _exact_penalties(case, s)
    if case["op"] == "clip":
        grads = [g.double() for g in s["grads"]]
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g) for g in grads]))
        factor = min(1.0, MAX_NORM / (float(norm) + EPS))
        return {"norm": norm, "grads": [g.mul_(factor) for g in grads]}
    # the gradients by differentiation of the forward formula
    f = torch.nn.functional
    act = {"none": lambda x: x, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda x: f.gelu(x, approximate="tanh"),
           "silu": f.silu}[case["act"]]
    leaves = [s["a"].double(), s["w"].double()] + ([s["bias"].double()] if case["bias"] else [])
    for leaf in leaves:
        leaf.requires_grad_(case["train"])
    out = act(f.linear(*leaves))
    out = out + s["residual"].double() if case["residual"] else out
    if not case["train"]:
        return out
    grads = torch.autograd.grad(out, leaves, s["dc"].double())
    return {"c": out.detach(), **dict(zip(("da", "dw", "dbias"), grads))}
