"""64-bit references of the language-model operators and the error bounds
their fp32 sums, planes and roundings allow, from the arithmetic alone.

Units: an fp32 addition or multiplication is off by at most 2^-24 of its
result; the matrix cores' internal additions may truncate, so each of theirs
counts 2^-23.  A rounding to a type is off by half of torch.finfo(t).eps."""
import torch

F64 = torch.float64
ADD = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# -- gemm_nt_q4 --------------------------------------------------------------

def q4_weights(q, scales, zeros, k, group):
    codes = torch.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1)[:, :k].to(F64)
    t = torch.arange(k, device=q.device) // group
    z = zeros.to(F64)[:, t] if zeros is not None else torch.tensor(8.0, dtype=F64, device=q.device)
    return (codes - z) * scales.to(F64)[:, t]


def q4(a, q, scales, zeros, group):
    """(exact, bound).  A term passes at most 96 additions of three 32-term matrix products,
    one per 32 k of its wave's slice, the 16 waves' and the product with its scale; three bf16
    planes of an fp32 activation leave out 2^-24 of it."""
    k = a.shape[1]
    w = q4_weights(q, scales, zeros, k, group)
    a64 = a.to(F64)
    exact = a64 @ w.t()
    size = a64.abs() @ w.abs().t()
    e = (96 + k / 32 + 16 + 2) * ADD * size
    if a.dtype == torch.float32:
        e = e + 2.0 ** -24 * size
    return exact, e + half_step(a.dtype) * (exact.abs() + e) + torch.finfo(a.dtype).tiny


# -- linear_cross_entropy ----------------------------------------------------

def plane_loss(planes):
    """What a product of two values in two fp16 planes leaves out, relative: both remainders
    (2^-11 for each of two roundings) and the product of the second planes (2^-22 again), and
    second-order terms; nothing of one plane, which is the value itself."""
    return 0.0 if planes == 1 else 3.1 * 2.0 ** -22


def sum_error(k, planes):
    """Additions a term of a tile product passes: the 32-deep matrix instructions of all
    plane products, one after another, and 32 inside one."""
    products = {1: 1, 2: 3}[planes]
    return (2 * -(-k // 64) * products + 32) * ADD + plane_loss(planes)


LAST = 2.0 ** -38  # last bit of a second plane, half of it, to its row's largest (2^13 units)


def cross_entropy(x, w, target, ignore, dloss):
    """dict of exact values and bounds: loss, lse, dx, dw.  fp32 runs as two fp16 planes, each
    row of x and w to its own largest value, g to the largest value the call could have."""
    planes = 1 if x.dtype == torch.bfloat16 else 2
    n, d = x.shape
    v = w.shape[0]
    keep = ((target != ignore) & (target >= 0) & (target < v)).nonzero()[:, 0]
    rows, w64, t = x[keep].to(F64), w.to(F64), target[keep]
    at = torch.arange(len(keep), device=x.device)
    z = rows @ w64.t()
    ez = (rows.abs() @ w64.abs().t()) * sum_error(d, planes)
    top_x, top_w = rows.abs().amax(1, keepdim=True), w64.abs().amax(1, keepdim=True)
    if planes == 2:
        ez = ez + LAST * (top_x * w64.abs().sum(1) + rows.abs().sum(1, keepdim=True) * top_w.t())
    lse_k = torch.logsumexp(z, 1)
    loss_k = lse_k - z[at, t]
    # exp's argument: a subtraction and a product (2^-24 each of its size) and exp2's own
    # 2^-23; the sum's additions: 16 of a lane, 2 shuffles, 4 waves, v/(64*32) tiles, 32 and 8,
    # or (few rows of fp32) v/1024 of a wave, 1024/32 of a thread and 32
    spread = (z.amax(1) - z.amin(1)) + 2 * ez.amax(1)
    adds = (66 + v / 1024) * 2.0 ** -24
    e_exp = spread * 2.0 ** -22 + 2.0 ** -22
    e_lse = ez.amax(1) + adds + 4 * e_exp + 2.0 ** -22 * lse_k.abs() + 2.0 ** -22
    e_loss = e_lse + ez[at, t] + 2.0 ** -23 * loss_k.abs()
    out = {"loss": torch.zeros(n, dtype=F64, device=x.device)}
    for name, val in (("lse", lse_k), ("e_lse", e_lse), ("e_loss", e_loss)):
        out[name] = torch.zeros(n, dtype=F64, device=x.device)
        out[name][keep] = val
    out["loss"][keep] = loss_k
    if dloss is None:
        return out
    p = torch.exp(z - lse_k[:, None])
    dl = dloss.to(F64)[keep][:, None]
    onehot = torch.zeros_like(p)
    onehot[at, t] = 1
    g = (p - onehot) * dl
    rel = torch.expm1(ez + e_lse[:, None] + (z - lse_k[:, None]).abs() * 2.0 ** -22 + 2.0 ** -22)
    eg = (p * rel + (p + onehot) * 2.0 ** -23) * dl.abs()
    eg = eg + (g.abs() + eg) * (2.0 ** -8 if planes == 1 else 2.0 ** -22)  # its planes
    ex = ew = 0
    if planes == 2 and len(keep):
        # g 2^c / (powers of the rows) has 2^-25 as half of its last bit and 2^12 at least where
        # its largest possible value is; the powers are 2^13 to 2^14 of their rows' largest
        most = (dl.abs() * top_x).amax() * top_w.amax()
        eg = eg + 2.0 ** -37 * 4 * most / (top_x * top_w.t()).clamp(min=1e-300)
        ex, ew = LAST * top_x, LAST * top_w
    se_v, se_n = sum_error(v, planes), sum_error(len(keep), planes)
    dx, dw = torch.zeros_like(x, dtype=F64), g.t() @ rows
    e_dx = torch.zeros_like(dx)
    dx[keep] = g @ w64
    ga = g.abs() + eg
    e_dx[keep] = eg @ w64.abs() + ga @ (w64.abs() * (se_v + (16 + v / 2048) * ADD) + ew)
    e_dw = eg.t() @ rows.abs() + ga.t() @ (rows.abs() * (se_n + 16 * ADD) + ex)
    step, tiny = half_step(x.dtype), torch.finfo(x.dtype).tiny
    out["dx"], out["dw"] = dx, dw
    out["e_dx"] = e_dx + step * (dx.abs() + e_dx) + tiny
    out["e_dw"] = e_dw + step * (dw.abs() + e_dw) + tiny
    return out


# -- newton_schulz -----------------------------------------------------------

def newton_schulz(g, steps, coeffs, eps):
    """(exact, bound on the Frobenius norm of the error) of one matrix.

    X is rounded to two fp16 planes (2^-22 of each value, and 2^-38 of the largest there can
    be); A = X X^T and B = b A + c A A to two for fp32 and one (2^-11, 2^-27) for bf16, whose
    products take X's first plane too (of more than 256 rows); products are off by sum_error of the products of
    absolute values besides.  An error of X before a step grows in that step by at most the
    operator norm of the step's derivative, which for an odd polynomial p of the singular
    values is the largest of |p(s) - p(t)| / |s - t| and |p(s) + p(t)| / (s + t) over pairs of
    them (|p'| where they meet); the singular values are taken with 1 % to spare, for the terms
    of second order."""
    a, b, c = coeffs
    one = g.dtype == torch.bfloat16 and min(g.shape) > 256
    keep = 2.0 ** -11 if one else 2.0 ** -22  # of A, B, and of what a product takes of X
    last = 2.0 ** -26 if one else LAST  # to the largest possible value (2^12 units at least)
    wide, add_k = 2.0 ** -22, (lambda k: sum_error(k, 1 if one else 2))
    taken = 2.1 * keep if one else 0.0  # sum_error has it for two planes
    x = g.to(F64)
    if x.shape[0] > x.shape[1]:
        x = x.t()
    x = x / (x.norm() + eps)
    r, k = x.shape
    err = x.norm() * (wide + 2.0 ** -22) + LAST * (r * k) ** 0.5
    bound = 1.0  # of X's singular values, as the call takes it
    for _ in range(steps):
        grid = torch.arange(1, 4097, dtype=F64) / 4096 * bound
        top_b = float((b * grid ** 2 + c * grid ** 4).abs().amax()) * 1.02
        s = torch.linalg.svdvals(x) * 1.01
        p = a * s + b * s ** 3 + c * s ** 5
        slope = (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().amax()
        ds, dp = s[:, None] - s[None], p[:, None] - p[None]
        diff = torch.where(ds.abs() > 1e-6, dp / torch.where(ds.abs() > 1e-6, ds, 1.0), 0.0)
        add = (p[:, None] + p[None]) / (s[:, None] + s[None] + 1e-300)
        grow = max(slope, diff.abs().amax(), add.abs().amax())
        if k > r:  # the rows' space beyond: p(s) / s
            grow = max(grow, (p / (s + 1e-300)).abs().amax())
        aa = x @ x.t()
        lost = last * bound * (r * k) ** 0.5  # of X's first plane or both, as a matrix
        e_a = (add_k(k) + taken) * (x.abs() @ x.abs().t()).norm() + 2.1 * s[0] * lost + \
            keep * aa.norm() + last * bound ** 2 * r
        e_aa = add_k(r) * (aa.abs() @ aa.abs()).norm() + 2.1 * s[0] ** 2 * e_a
        bb = b * aa + c * aa @ aa
        e_b = abs(b) * e_a + abs(c) * e_aa + (keep + 3 * 2.0 ** -24) * (
            abs(b) * aa.abs() + abs(c) * aa.abs() @ aa.abs()).norm() + last * top_b * r
        nxt = a * x + bb @ x
        local = s[0] * e_b + (add_k(r) + taken) * (bb.abs() @ x.abs()).norm() + top_b * lost + (
            wide + 3 * 2.0 ** -24) * (abs(a) * x.abs() + (bb @ x).abs()).norm()
        bound = float((a * grid + b * grid ** 3 + c * grid ** 5).abs().amax()) * 1.02
        err = grow * err + local + LAST * bound * (r * k) ** 0.5
        x = nxt
    err = err + half_step(g.dtype) * (x.norm() + err)
    return (x.t() if g.shape[0] > g.shape[1] else x), err


# -- logit_penalties ---------------------------------------------------------

def logit_penalties(z, tokens, lengths, prompts, repetition, frequency, presence, bias, mask):
    """(exact, bound), a row and a token at a time on the host.  Each of up to five operations
    rounds to fp32 (2^-24 of its result, to which the sizes of all terms are a bound; half of
    the smallest subnormal), the end to the type."""
    n, v = z.shape
    x = z.to(F64).cpu()
    size = torch.zeros_like(x)
    host = lambda t: None if t is None else t.cpu()  # noqa: E731
    tokens, lengths, prompts, repetition, frequency, presence, bias, mask = map(
        host, (tokens, lengths, prompts, repetition, frequency, presence, bias, mask))
    for i in range(n):
        seen, made = {}, {}
        if tokens is not None:
            t = tokens.shape[1]
            stop = t if lengths is None else min(max(int(lengths[i]), 0), t)
            for p, tok in enumerate(tokens[i, :stop].tolist()):
                if 0 <= tok < v:
                    seen[tok] = True
                    if p >= (0 if prompts is None else int(prompts[i])):
                        made[tok] = made.get(tok, 0) + 1
        for tok in seen:
            if repetition is not None:
                r = float(repetition[i])
                x[i, tok] = x[i, tok] / r if x[i, tok] > 0 else x[i, tok] * r
            if tok in made:
                for by in ([] if frequency is None else [float(frequency[i]) * made[tok]]) + (
                        [] if presence is None else [float(presence[i])]):
                    size[i, tok] += x[i, tok].abs() + abs(by)
                    x[i, tok] -= by
            size[i, tok] += x[i, tok].abs()
        if bias is not None:
            b = bias if bias.dim() == 1 or bias.shape[0] == 1 else bias[i]
            size[i] += x[i].abs() + b.reshape(-1).abs()
            x[i] += b.reshape(-1).to(F64)
        if mask is not None:
            m = mask if mask.dim() == 1 or mask.shape[0] == 1 else mask[i]
            words = m.reshape(-1).tolist()
            for j in range(v):
                if not words[j // 32] >> (j % 32) & 1:
                    x[i, j], size[i, j] = float("-inf"), 0
    over = x.to(z.dtype).isinf()  # (past the type's range)
    x[over] = x[over].sign() * float("inf")
    e = size * 2.0 ** -24 * 1.01 + 2.0 ** -148
    e = e + half_step(z.dtype) * (x.abs() + e) + torch.finfo(z.dtype).smallest_normal * torch.finfo(z.dtype).eps
    return x, e


# -- gemm_nt_epi -------------------------------------------------------------

def activation(x, act):
    """act(x), act'(x) in 64 bits, with their limits at infinity."""
    if act is None:
        return x, torch.ones_like(x)
    inf = torch.where(x.isnan(), x, torch.full_like(x, float("nan")))
    flat = x.clamp(-300, 300)  # (both are their limits in fp32 from 120 on)
    if act == "relu":
        y, d = x.clamp(min=0), (x > 0).to(x.dtype)
        return torch.where(x.isnan(), inf, y), torch.where(x.isnan(), inf, d)
    if act == "gelu":
        below = 0.5 * torch.erfc(-flat * 0.5 ** 0.5)
        d = below + flat * torch.exp(-flat * flat / 2) / (2 * torch.pi) ** 0.5
    elif act == "gelu_tanh":
        c = 2 * (2 / torch.pi) ** 0.5
        u = c * (flat + 0.044715 * flat ** 3)
        below = torch.sigmoid(u)
        d = below + flat * below * torch.sigmoid(-u) * c * (1 + 3 * 0.044715 * flat ** 2)
    else:
        below = torch.sigmoid(flat)
        d = below + flat * below * torch.sigmoid(-flat)
    y = torch.where(x > 300, x, flat * below)
    return torch.where(x.isnan(), inf, y), d


STEEP = 1.13  # no activation's slope is larger, nor (by a little) any second derivative's size


def act_error(x, e, act):
    """Of act(v) and act'(v) in fp32 for |v - x| <= e: the slope times e, and evaluation.  Every
    value is a product of at most x and factors whose relative error is 2^-22 for each of a few
    operations and, of the exponential, 2^-23 for each unit of its argument (at most x^2 / 2 or
    1.6 (x + 0.045 x^3), where the value has not vanished: 110)."""
    if act is None:
        return e, torch.zeros_like(e)
    y, d = activation(x, act)
    if act == "relu":
        return e, torch.where(x.abs() <= e, torch.ones_like(e), torch.zeros_like(e))
    arg = (4 + torch.minimum(x.abs() * 2 + x * x, torch.full_like(x, 110.0))) * 2.0 ** -22
    arg = arg.nan_to_num()
    small = (y.abs() + d.abs()).clamp(max=2.0) + torch.exp(-x.abs().clamp(max=90) * 0.5)
    return STEEP * e + arg * (y.abs() + 2.0 ** -120), STEEP * e + arg * small


def product_error(a64, b64, dtype):
    """Bound on the error of a @ b.T of two matrices of a type (in 64 bits here) by the tile product
    or the few rows' kernel: sum_error and up to 16 parts' joining; fp32 to each row's 2^-38
    besides."""
    planes, k = 2 if dtype == torch.float32 else 1, a64.shape[1]
    e = (a64.abs() @ b64.abs().t()) * (sum_error(k, planes) + 40 * ADD)
    if planes == 2 and k:
        ta, tb = a64.abs().amax(1, keepdim=True), b64.abs().amax(1, keepdim=True)
        e = e + LAST * (ta * b64.abs().sum(1) + a64.abs().sum(1, keepdim=True) * tb.t())
        e = e + 2.0 ** -148
    return e


def rounded(x, e, dtype):
    """The bound after a rounding to dtype."""
    info = torch.finfo(dtype)
    return e + half_step(dtype) * (x.abs() + e) + info.smallest_normal * info.eps


def gemm_epi(a, w, bias, act, residual):
    """dict of exact values and bounds: pre, c."""
    v = a.to(F64) @ w.to(F64).t()
    e = product_error(a.to(F64), w.to(F64), a.dtype)
    if bias is not None:
        v = v + bias.to(F64)
        e = e + 2.0 ** -24 * (v.abs() + e)
    y, _ = activation(v, act)
    ey, _ = act_error(v, e, act)
    if residual is not None:
        y = y + residual.to(F64)
        ey = ey + 2.0 ** -24 * (y.abs() + ey)
    return {"pre": v, "e_pre": rounded(v, e, a.dtype), "c": y, "e_c": rounded(y, ey, a.dtype)}


def gemm_epi_grad(dc, a, w, pre, act):
    """dict of exact values for this pre, and bounds: da, dw, dbias.  16-bit types round dP to the
    type (its largest subnormal's half step, twice in fp16, which may hold halves); up to 128 rows
    with a second matrix of what that leaves, whose own rounding is half a step of half a step."""
    dc64, a64, w64 = dc.to(F64), a.to(F64), w.to(F64)
    dp, edp = dc64, torch.zeros_like(dc64)
    if act is not None:
        x = pre.to(F64)
        _, d = activation(x, act)
        _, ed = act_error(x, torch.zeros_like(x), act)
        dp = dc64 * d
        edp = dc64.abs() * ed + 2.0 ** -24 * (dp.abs() + dc64.abs() * ed) + 2.0 ** -149
    held = edp
    info = torch.finfo(dc.dtype)
    if act is not None and dc.dtype != torch.float32:
        step = half_step(dc.dtype) ** (2 if len(dc) <= 128 else 1)
        held = edp + step * (dp.abs() + edp) + 2 * info.smallest_normal * info.eps
    out = {"da": dp @ w64, "dw": dp.t() @ a64, "dbias": dp.sum(0)}
    e_da = held @ w64.abs() + product_error(dp, w64.t(), dc.dtype) * 1.01
    e_dw = held.t() @ a64.abs() + product_error(dp.t(), a64.t(), dc.dtype) * 1.01
    e_db = edp.sum(0) + 22 * 2.0 ** -24 * (dp.abs() + edp).sum(0)
    for name, e in (("da", e_da), ("dw", e_dw), ("dbias", e_db)):
        out["e_" + name] = rounded(out[name], e, dc.dtype)
    return out
