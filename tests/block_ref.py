"""Plain float64 forms of a transformer block's layers, written from their definitions with torch on
the CPU, and the bounds that the arithmetic of the library's kernels gives for each value.

u is the unit roundoff of the output type (one rounding), e = 2^-24 that of fp32.  A rounding is off by
u |y|, but at least by half the spacing of the type's smallest numbers: fp16 holds multiples of 2^-24 below 2^-14."""

import math

import torch

from layers_ref import U

E = 2.0 ** -24
LEAST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def rounding(y, dtype):
    return (U[dtype] * y.abs()).clamp(min=LEAST[dtype])


# ------------------------------------------------------------------ layer norm
def layer_norm_fwd(x, gamma, beta, eps):
    """y, mean, rstd and their bounds."""
    u, t, c = U[x.dtype], x.dtype, x.shape[1]
    x = x.double()
    ga = torch.ones(c, dtype=torch.float64) if gamma is None else gamma.double()
    be = torch.zeros(c, dtype=torch.float64) if beta is None else beta.double()
    mean = x.mean(1)
    rstd = (((x - mean[:, None]) ** 2).mean(1) + eps) ** -0.5
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * ga + be
    h = (c / 512 + 64) * E  # additions that follow one another, and the joins
    mb = h * x.abs().mean(1)
    # the variance is summed around the rounded mean: off by its square besides
    rb = rstd * (h + (mb * rstd) ** 2 + 4 * E)
    xb = (mb * rstd)[:, None] + 4 * E * (x - mean[:, None]).abs() * rstd[:, None] + xh.abs() * (rb / rstd)[:, None]
    return (y, mean, rstd), (rounding(y, t) + (1 + u) * (xb * ga.abs() + 3 * E * (xh * ga).abs() + E * y.abs()), mb + E * mean.abs(), rb)


def layer_norm_bwd(dy, x, gamma, mean, rstd):
    """dx, dgamma, dbeta and their bounds, from the given statistics."""
    u, t, (n, c) = U[x.dtype], x.dtype, x.shape
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    ga = torch.ones(c, dtype=torch.float64) if gamma is None else gamma.double()
    xh = (x - mean) * rstd
    w = dy * ga
    a, b = w.mean(1, keepdim=True), (w * xh).mean(1, keepdim=True)
    dx = rstd * (w - a - xh * b)
    h = (c / 512 + 64) * E
    xb = 3 * E * xh.abs()  # one difference, one product
    ab = h * w.abs().mean(1, keepdim=True)
    bb = h * (w * xh).abs().mean(1, keepdim=True) + (w.abs() * xb).mean(1, keepdim=True)
    d = 2 * E * w.abs() + ab + xh.abs() * bb + xb * b.abs() + 4 * E * (w.abs() + a.abs() + (xh * b).abs())
    k = (n / 100 + 64) * E
    return ((dx, (dy * xh).sum(0), dy.sum(0)),
            (rounding(dx, t) + (1 + u) * rstd * d, k * (dy * xh).abs().sum(0) + (dy.abs() * xb).sum(0), k * dy.abs().sum(0)))


# ------------------------------------------------------------ rotary positions
def rope(x, coords, pairs, base, back=False):
    u, t = U[x.dtype], x.dtype
    x = x.double()
    y, bound = x.clone(), torch.zeros_like(x)
    i = 0
    for axis in range(3):
        for j in range(pairs[axis]):
            angle = coords[:, 1 + axis].double() * base ** (-j / pairs[axis])
            c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if back else 1)
            a, b = x[:, :, 2 * i], x[:, :, 2 * i + 1]
            y[:, :, 2 * i], y[:, :, 2 * i + 1] = a * c - b * s, a * s + b * c
            # sine and cosine to 2^-22 (float64's own angle is off by 2^-53 of itself), two products, a sum
            off = (2.0 ** -22 + 2.0 ** -52 * angle.abs())[:, None]
            for k in (2 * i, 2 * i + 1):
                bound[:, :, k] = (1 + u) * (a.abs() + b.abs()) * (off + 3 * E) + rounding(y[:, :, k], t)
            i += 1
    return y, bound


# ----------------------------------------------------------- routing to experts
def scores(logits, score):
    """Scores in float64, and which experts there are."""
    z = logits.double()
    there = z > -math.inf  # NaN is not
    z = torch.where(there, z.clamp(max=float(torch.finfo(torch.float32).max)), -math.inf)
    if score == "sigmoid":
        return torch.where(there, torch.sigmoid(z), 0.0), there, z
    most = z.max(1, keepdim=True).values
    e = torch.where(there, torch.exp(z - torch.where(most > -math.inf, most, 0.0)), 0.0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300), there, z


def route_fwd(logits, top_k, score, bias, groups, top_groups, renorm, scale):
    p, there, z = scores(logits, score)
    n, experts = p.shape
    c = z if bias is None and groups == 1 else p + (0.0 if bias is None else bias.double())
    c = torch.where(there, c, -math.inf)
    expert = torch.full((n, top_k), -1, dtype=torch.int32)
    gate = torch.zeros(n, top_k, dtype=torch.float64)
    size = experts // groups
    for r in range(n):
        row = c[r].tolist()
        if groups > 1:
            best = []
            for g in range(groups):
                own = sorted((v for v in row[g * size:(g + 1) * size] if v > -math.inf), reverse=True)[:2]
                best.append(sum(own) if own else -math.inf)
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            row = [row[e] if e // size in kept and best[e // size] > -math.inf else -math.inf for e in range(experts)]
        chosen = [e for e in sorted(range(experts), key=lambda e: (-row[e], e))[:top_k] if row[e] > -math.inf]
        w = [float(p[r, e]) for e in chosen]
        if renorm and chosen:
            log = [float(torch.nn.functional.logsigmoid(z[r, e])) if score == "sigmoid" else float(z[r, e]) for e in chosen]
            w = [math.exp(v - max(log)) for v in log]
            w = [v / sum(w) for v in w]
        expert[r, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        gate[r, :len(chosen)] = scale * torch.tensor(w, dtype=torch.float64)
    # exp to 2 ulp of an argument rounded once (up to 104 of them matter), a sum of at most experts / 32 + 40 steps
    return (expert, gate), gate.abs() * ((experts / 32 + 48) * E + 2 * E * 104) + 1e-37


def route_bwd(dgate, logits, expert, score, renorm, scale):
    u = U[logits.dtype]
    p, there, z = scores(logits, score)
    n, experts = p.shape
    dl, mag = torch.zeros_like(p), torch.zeros_like(p)
    for r in range(n):
        own = [(int(e), float(g)) for e, g in zip(expert[r], dgate[r]) if e >= 0 and there[r, int(e)]]
        if not own:
            continue
        if renorm:
            log = [float(torch.nn.functional.logsigmoid(z[r, e])) if score == "sigmoid" else float(z[r, e]) for e, _ in own]
            w = [math.exp(v - max(log)) for v in log]
            w = [v / sum(w) for v in w]
        else:
            w = [float(p[r, e]) for e, _ in own]
        dot = sum(a * g for a, (_, g) in zip(w, own)) if renorm or score == "softmax" else 0.0
        size = sum(a * abs(g) for a, (_, g) in zip(w, own))
        if score == "softmax" and not renorm:
            dl[r] -= scale * p[r] * dot
            mag[r] += scale * p[r] * size
        for a, (e, g) in zip(w, own):
            slope = float(torch.sigmoid(-z[r, e])) if score == "sigmoid" else 1.0
            dl[r, e] += scale * a * slope * (g - (dot if renorm else 0.0))
            mag[r, e] += scale * a * slope * (abs(g) + size)
    return dl, rounding(dl, logits.dtype) + (1 + u) * mag * ((experts / 32 + 64) * E + 2 * E * 104) + 1e-37


# -------------------------------------------------------------------- attention
def segment_rows(seg, s):
    return slice(int(seg[s]), int(seg[s + 1]))


def attention_fwd(q, k, v, seg, seg_k, scale, rounded):
    """o, lse and their bounds.  rounded: probabilities are rounded to the inputs' type before the product."""
    u, t = U[q.dtype], q.dtype
    q, k, v = q.double(), k.double(), v.double()
    (nq, hq, d), hk = q.shape, k.shape[1]
    o, lse = torch.zeros_like(q), torch.full((nq, hq), -math.inf, dtype=torch.float64)
    ob, lb = torch.zeros_like(q), torch.zeros(nq, hq, dtype=torch.float64)
    for s in range(len(seg) - 1):
        a, b = segment_rows(seg, s), segment_rows(seg_k, s)
        m = b.stop - b.start
        if a.stop <= a.start or m <= 0:
            continue
        for h in range(hq):
            g = h // (hq // hk)
            z = scale * q[a, h] @ k[b, g].T
            lse[a, h] = torch.logsumexp(z, 1)
            p = torch.softmax(z, 1)
            o[a, h] = p @ v[b, g]
            # scores: d products and sums in fp32, then one product with scale log2 e and the subtraction
            off = ((d + 4) * 2 * E * scale * (q[a, h].abs() @ k[b, g].abs().T) + 4 * E * (z.abs() + 1)).amax(1)
            near = 2 * off + (2 * m + 64) * E + 2.0 ** -20
            lb[a, h] = near + 4 * E * lse[a, h].abs()
            size = p @ v[b, g].abs()
            if rounded and t is torch.float16:
                # the largest probability is kept as 2^7 or more, the smallest ones as multiples of 2^-24
                ob[a, h] += 2.0 ** -32 * v[b, g].abs().sum(0)
            ob[a, h] += size * (near + (m + 64) * 2 * E + (u if rounded else 0.0))[:, None]
    return (o, lse), (ob * (1 + u) + rounding(o, t) + 2.0 ** -30, lb)


def attention_bwd(dout, q, k, v, o, lse, seg, seg_k, scale, rounded):
    """dq, dk, dv and their bounds, from the given o and lse."""
    u, t = U[q.dtype], q.dtype
    r = u if rounded else 0.0
    dout, q, k, v, o, lse = (x.double() for x in (dout, q, k, v, o, lse))
    (nq, hq, d), hk = q.shape, k.shape[1]
    out = [torch.zeros_like(x) for x in (q, k, v)]
    bound = [torch.zeros_like(x) for x in (q, k, v)]
    for s in range(len(seg) - 1):
        a, b = segment_rows(seg, s), segment_rows(seg_k, s)
        n, m = a.stop - a.start, b.stop - b.start
        if n <= 0 or m <= 0:
            continue
        for h in range(hq):
            g = h // (hq // hk)
            z = scale * q[a, h] @ k[b, g].T
            p = torch.exp(z - lse[a, h, None])
            off = (d + 4) * 2 * E * scale * (q[a, h].abs() @ k[b, g].abs().T) + 4 * E * (z.abs() + lse[a, h, None].abs() + 1) + 2.0 ** -20
            dp, delta = dout[a, h] @ v[b, g].T, (dout[a, h] * o[a, h]).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dpb = (d + 4) * 2 * E * (dout[a, h].abs() @ v[b, g].abs().T + (dout[a, h] * o[a, h]).abs().sum(1, keepdim=True))
            dsb = ds.abs() * (r + off + 4 * E) + p * dpb * (1 + off)
            pb = p * (r + off)
            if rounded and t is torch.float16:
                # p is kept times 2^14 and ds times 2^14 / 2^e with 2^(e - 1) <= 2 max|do| max|v|, the smallest as
                # multiples of 2^-24
                pb = pb + 2.0 ** -39
                dsb = dsb + 2.0 ** -38 * 2 * dout.norm(dim=2).max() * v.norm(dim=2).max()
            grow = lambda count: (count * (hq // hk) + 64) * 2 * E  # noqa: E731
            out[0][a, h] += scale * ds @ k[b, g]
            bound[0][a, h] += scale * (dsb + grow(m) * ds.abs()) @ k[b, g].abs()
            out[1][b, g] += scale * ds.T @ q[a, h]
            bound[1][b, g] += scale * (dsb + grow(n) * ds.abs()).T @ q[a, h].abs()
            out[2][b, g] += p.T @ dout[a, h]
            bound[2][b, g] += (pb + grow(n) * p).T @ dout[a, h].abs()
    return out, [(1 + u) * y + rounding(x, t) + 2.0 ** -30 for x, y in zip(out, bound)]
