"""The operators of a transformer block over voxels, one at a time.

Rows of a batch lie in one [n, C] matrix, each row a voxel or a token; `seg` [S + 1]
holds the offsets of the samples (or windows) among them.

  norm     layer norm of each row, forward and backward
  rope     rotary positions from the voxels' (b, z, y, x) coordinates, each axis with
           frequencies of its own, and the gradient (the rotation back)
  route    the experts of each token: softmax or sigmoid scores, a bias that counts in
           the choice only, groups of experts, the best k and their weights; and the
           gradient by the logits
  attn     attention of a segment's queries to the same segment's keys, forward and
           backward (the probabilities computed again from the forward's log-sum)

`listed()` and `draw()` give cases, `prepare()` a case's inputs, `run()` one
pass: the plain form in 32 bits, or the library's kernels where `own` is true.
`work()` counts what a pass has to move and compute; `exact()` is the definition
in 64 bits.
"""

import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
BASE = 10000.0
EXACT_FLOPS = 1.2e13      # what 64 bits take some ten seconds for
PADDED = 2 ** 28          # scores that the plain form holds at once


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # the 32^3 set of one sample: the smallest call, where latency counts
        dict(name="norm_fwd_2k_f32", op="norm", pass_="fwd", n=2000, c=16, type="f32"),
        # the 4 x 192^3 shells of the training step
        dict(name="norm_bwd_shells_bf16", op="norm", pass_="bwd", n=498145, c=64, type="bf16"),
        # queries and keys of the 256^3 shell's strided voxels, inside the projection's rows
        dict(name="rope_fwd_shell_bf16", op="rope", pass_="fwd", n=99569, heads=16, d=64,
             pz=10, py=11, px=11, extra=8, extent=256, type="bf16"),
        # an odd number of heads, channels that are not rotated, far cells
        dict(name="rope_bwd_odd_f32", op="rope", pass_="bwd", n=12345, heads=3, d=40,
             pz=5, py=6, px=7, extra=0, extent=1600, type="f32"),
        # two of 64 experts for 65,536 tokens
        dict(name="route_fwd_64_bf16", op="route", pass_="fwd", n=65536, experts=64, k=2, score="softmax",
             bias=False, groups=1, kept=1, renorm=True, scale=1.0, type="bf16"),
        # eight of 256, from the four best of eight groups
        dict(name="route_fwd_groups_f32", op="route", pass_="fwd", n=16000, experts=256, k=8, score="sigmoid",
             bias=True, groups=8, kept=4, renorm=True, scale=2.5, type="f32"),
        # a training step's gradient, for weights that are not renormalised
        dict(name="route_bwd_64_bf16", op="route", pass_="bwd", n=65536, experts=64, k=2, score="softmax",
             bias=False, groups=1, kept=1, renorm=False, scale=1.0, type="bf16"),
        # the 2,000-voxel set in full fp32
        dict(name="attn_fwd_2k_f32", op="attn", pass_="fwd", nq=2000, nk=2000, segments=1, cross=False,
             hq=4, hk=4, d=16, type="f32"),
        # four samples of a coarse level
        dict(name="attn_fwd_samples_bf16", op="attn", pass_="fwd", nq=32768, nk=32768, segments=4, cross=False,
             hq=8, hk=8, d=64, type="bf16"),
        # one query for each sample, over all its voxels; four query heads share their keys
        dict(name="attn_fwd_query_bf16", op="attn", pass_="fwd", nq=4, nk=498145, segments=4, cross=True,
             hq=8, hk=2, d=64, type="bf16"),
        # the largest: a training step over long samples with wide heads
        dict(name="attn_bwd_long_bf16", op="attn", pass_="bwd", nq=32768, nk=32768, segments=2, cross=False,
             hq=8, hk=8, d=128, type="bf16"),
        # the LiDAR batch in windows of some 200 voxels
        dict(name="attn_bwd_windows_f16", op="attn", pass_="bwd", nq=120000, nk=120000, segments=600, cross=False,
             hq=4, hk=4, d=32, type="f16"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "route", "route", "attn", "attn", "attn"])
    type_ = rng.choice(["f32", "f16", "bf16", "bf16"])
    pass_ = rng.choice(["fwd", "bwd"])
    if op == "norm":
        c = _spread(rng, 8, 4000)
        c = rng.choice([c, c // 8 * 8])
        return dict(op=op, pass_=pass_, n=_spread(rng, 100, 30000000 // c), c=c, type=type_)
    if op == "rope":
        d = rng.choice([16, 32, 40, 64, 96, 128])
        heads = rng.choice([1, 3, 4, 8, 16])
        third = rng.choice([d // 6, d // 8])
        return dict(op=op, pass_=pass_, n=_spread(rng, 1, 60000000 // (d * heads)), heads=heads, d=d,
                    pz=d // 2 - 2 * (d // 6), py=third, px=third, extra=rng.choice([0, heads]),
                    extent=rng.choice([32, 192, 1600]), type=type_)
    if op == "route":
        experts = rng.choice([4, 8, 16, 60, 64, 128, 160, 256])
        groups = rng.choice([1, 1, 4])
        kept = rng.choice([1, 2, 3]) if groups > 1 else 1
        return dict(op=op, pass_=pass_, n=_spread(rng, 1, 8000000 // experts), experts=experts,
                    k=rng.randint(1, min(8, experts // groups * kept)), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, kept=kept, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), type=type_)
    d = rng.choice([16, 32, 40, 64, 64, 80, 128])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 1, 2, 3, 4])
    if hq > 16:
        hq = hk
    segments = rng.choice([1, 2, 4, 21, 300])
    cross = rng.random() < 0.35
    most = 1.0e11 if type_ == "f32" else 1.5e12
    while True:
        nk = _spread(rng, max(segments, 16), 60000)
        nq = nk if not cross else rng.choice([segments, _spread(rng, segments, 60000)])
        if 10.0 * nq * nk / segments * d * hq <= most:
            return dict(op=op, pass_=pass_, nq=nq, nk=nk, segments=segments, cross=cross, hq=hq, hk=hk, d=d, type=type_)


# ----------------------------------------------------------------------- inputs
def _sizes(n, segments, salt):
    """Rows of each segment, some twice as many as others (the same for every seed)."""
    if n == segments:
        return [1] * n
    rng = random.Random(1000003 * n + 101 * segments + salt)
    weight = [rng.uniform(0.7, 1.4) for _ in range(segments)]
    edge, total, sizes, done = 0.0, sum(weight), [], 0
    for w in weight:
        edge += w
        upto = int(round(n * edge / total))
        sizes.append(upto - done)
        done = upto
    return sizes


def _offsets(sizes):
    seg = torch.zeros(len(sizes) + 1, dtype=torch.int32)
    seg[1:] = torch.tensor(sizes).cumsum(0)
    return seg.cuda()


def _attn_sizes(case):
    return _sizes(case["nq"], case["segments"], 0), _sizes(case["nk"], case["segments"], 1 if case["cross"] else 0)


def _pairs(case):
    """Turned pairs of channels of each axis (z, y, x)."""
    return [case["pz"], case["py"], case["px"]]


def _steps(pairs):
    """Radians a cell, of each axis' pairs one after the other."""
    return torch.cat([BASE ** (-torch.arange(p, dtype=torch.float64) / max(p, 1)) for p in pairs])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, back = case["op"], case["pass_"] == "bwd"

    def normal(*shape, std=1.0, type_=None):
        a = torch.randn(*shape, generator=gen, device="cuda") * std
        return a.to(TYPES[type_ or case["type"]])

    state = dict(case=case)
    if op == "norm":
        n, c = case["n"], case["c"]
        # the residual stream: every channel with a mean and a spread of its own
        x = torch.randn(n, c, generator=gen, device="cuda")
        x = x * torch.empty(c, device="cuda").uniform_(0.5, 2.0, generator=gen) + normal(c, type_="f32")
        state.update(x=x.to(TYPES[case["type"]]), gamma=1 + normal(c, std=0.2, type_="f32"),
                     beta=normal(c, std=0.2, type_="f32"))
        if back:
            state["dy"] = normal(n, c)
            state["mean"], state["rstd"] = _plain_stats(state["x"])
    elif op == "rope":
        n, heads = case["n"], case["heads"]
        x = normal(n, heads + case["extra"], case["d"])
        coords = torch.randint(0, case["extent"], (n, 4), generator=gen, device="cuda", dtype=torch.int32)
        coords[:, 0] = torch.arange(n, device="cuda") * 2 // n
        state.update(x=x[:, :heads], coords=coords, freq=_steps(_pairs(case)).cuda())
        if own:
            import sparse_convolution_hash_gb300 as spc

            state["steps"] = spc.spc_rope_steps(_pairs(case), BASE)
    elif op == "route":
        n, experts = case["n"], case["experts"]
        favour = normal(experts, std=0.5, type_="f32")
        state["logits"] = (normal(n, experts, std=1.2, type_="f32") + favour).to(TYPES[case["type"]])
        state["bias"] = normal(experts, std=0.05, type_="f32") if case["bias"] else None
        if back:
            state["expert"] = _plain_choice(state)[0].to(torch.int32)
            state["dgate"] = normal(n, case["k"], type_="f32")
    else:
        hq, hk, d = case["hq"], case["hk"], case["d"]
        sizes_q, sizes_k = _attn_sizes(case)
        state.update(sizes_q=sizes_q, sizes_k=sizes_k, seg_q=_offsets(sizes_q),
                     seg_k=_offsets(sizes_k) if case["cross"] else None)
        if case["cross"]:
            state["q"] = normal(case["nq"], hq, d, std=1.5)
            kv = normal(case["nk"], 2 * hk, d)
            state["k"], state["v"] = kv[:, :hk], kv[:, hk:]
        else:  # slices of one projection's rows
            qkv = normal(case["nq"], hq + 2 * hk, d)
            qkv[:, :hq] *= 1.5
            state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        if back:
            state["do"] = normal(case["nq"], hq, d)
            kept = _plain_attn_fwd(state)
            state["o"], state["lse"] = kept["o"], kept["lse"]
    return state


# ------------------------------------------------------------------ plain forms
def _plain_stats(x):
    x = x.float()
    mean = x.mean(1)
    return mean, 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + EPS)


def _plain_norm(state):
    x = state["x"].float()
    if state["case"]["pass_"] == "fwd":
        mean, rstd = _plain_stats(x)
        y = (x - mean[:, None]) * rstd[:, None] * state["gamma"] + state["beta"]
        return {"y": y.to(state["x"].dtype), "mean": mean, "rstd": rstd}
    rstd = state["rstd"][:, None]
    xh = (x - state["mean"][:, None]) * rstd
    dy = state["dy"].float()
    u = dy * state["gamma"]
    dx = rstd * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    return {"dx": dx.to(state["x"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _plain_rope(state):
    case, x = state["case"], state["x"]
    pairs, turned = _pairs(case), 2 * sum(_pairs(case))
    axis = torch.tensor([1 + a for a in range(3) for _ in range(pairs[a])], device="cuda")
    angle = state["coords"][:, axis].double() * state["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["pass_"] == "bwd":
        sin = -sin
    a, b = x[:, :, 0:turned:2].float(), x[:, :, 1:turned:2].float()
    y = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    y[:, :, 0:turned:2] = a * cos - b * sin
    y[:, :, 1:turned:2] = a * sin + b * cos
    y[:, :, turned:] = x[:, :, turned:]
    return y.to(x.dtype)


def _plain_scores(state, type_):
    z = state["logits"].to(type_)
    if state["case"]["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_choice(state):
    """Chosen experts, best first, and all scores; in 64 bits, as a choice between near values hangs on the last."""
    case = state["case"]
    p = _plain_scores(state, torch.float64)
    c = p if state["bias"] is None else p + state["bias"].double()
    n, experts = c.shape
    if case["groups"] > 1:
        by = c.view(n, case["groups"], -1)
        best = by.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros(n, case["groups"], dtype=torch.bool, device="cuda").scatter_(1, order, True)
        c = torch.where(keep[:, :, None], by, -math.inf).view(n, experts)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]], p


def _plain_route(state):
    case = state["case"]
    if case["pass_"] == "fwd":
        expert, p = _plain_choice(state)
        gate = p.float().gather(1, expert)
        if case["renorm"]:
            gate = gate / gate.sum(1, keepdim=True)
        return {"expert": expert.to(torch.int32), "gate": gate * case["scale"]}
    p = _plain_scores(state, torch.float32)
    expert, dgate = state["expert"].long(), state["dgate"] * case["scale"]
    own_p = p.gather(1, expert)
    if case["renorm"]:
        total = own_p.sum(1, keepdim=True)
        dgate = (dgate - (dgate * own_p).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_(1, expert, dgate)
    dl = p * (1 - p) * dp if case["score"] == "sigmoid" else p * (dp - (own_p * dgate).sum(1, keepdim=True))
    return dl.to(state["logits"].dtype)


def _batches(state):
    """Segments that the plain form takes at once: all of them, padded, or one after the other."""
    case, (sq, sk) = state["case"], (state["sizes_q"], state["sizes_k"])
    if len(sq) * max(sq) * max(sk) * case["hq"] <= PADDED:
        return [list(range(len(sq)))]
    return [[s] for s in range(len(sq)) if sq[s]]


def _where(seg, sizes, at, heads):
    """Rows of the segments side by side [s, longest], and which of them there are."""
    first = seg[:-1].long()[at] if len(at) > 1 else seg[at[0]:at[0] + 1].long()
    longest = max(max(sizes[s] for s in at), 1)
    step = torch.arange(longest, device="cuda")
    count = (seg[1:] - seg[:-1]).long()[at] if len(at) > 1 else (seg[at[0] + 1:at[0] + 2] - seg[at[0]:at[0] + 1]).long()
    there = step < count[:, None]
    return torch.where(there, first[:, None] + step, 0), there


def _heads(x, rows, there, hk):
    """[s, hk, heads of a group * rows, d] in 32 bits, zeros where there is no row."""
    got = torch.where(there[:, :, None, None], x[rows].float(), 0.0)
    s, length, h, d = got.shape
    return got.view(s, length, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(s, hk, -1, d)


def _rows_of(x, s, hk, length):
    """Back to [s, rows, heads, d]."""
    d = x.shape[-1]
    return x.view(s, hk, -1, length, d).permute(0, 3, 1, 2, 4).reshape(s, length, -1, d)


def _plain_attn(state):
    return _plain_attn_fwd(state) if state["case"]["pass_"] == "fwd" else _plain_attn_bwd(state)


def _plain_attn_fwd(state):
    case = state["case"]
    q, k, v = state["q"], state["k"], state["v"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    seg_k = state["seg_q"] if state["seg_k"] is None else state["seg_k"]
    o = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, device="cuda")
    for at in _batches(state):
        rq, tq = _where(state["seg_q"], state["sizes_q"], at, hq)
        rk, tk = _where(seg_k, state["sizes_k"], at, hk)
        for h in [slice(0, hk)] if len(at) > 1 or rq.numel() * rk.numel() * hq <= PADDED else [slice(i, i + 1) for i in range(hk)]:
            hs, gs = h.stop - h.start, slice(h.start * (hq // hk), h.stop * (hq // hk))
            qs, ks, vs = _heads(q[:, gs], rq, tq, hs), _heads(k[:, h], rk, tk, hs), _heads(v[:, h], rk, tk, hs)
            s = qs @ ks.transpose(2, 3) * d ** -0.5
            s.masked_fill_(~tk[:, None, None, :], -math.inf)
            m = s.max(3, keepdim=True).values.clamp(min=-1e30)
            e = torch.exp(s - m)
            total = e.sum(3, keepdim=True)
            got = e @ vs / total.clamp(min=1e-38)
            log = torch.log(total) + torch.where(total > 0, m, 0.0)
            here = rq[tq]
            o[here, gs] = _rows_of(got, len(at), hs, rq.shape[1])[tq].to(o.dtype)
            lse[here, gs] = _rows_of(log, len(at), hs, rq.shape[1])[tq][:, :, 0]
    return {"o": o, "lse": lse}


def _plain_attn_bwd(state):
    case = state["case"]
    q, k, v = state["q"], state["k"], state["v"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    scale = d ** -0.5
    seg_k = state["seg_q"] if state["seg_k"] is None else state["seg_k"]
    dq, dk, dv = (torch.zeros(x.shape, dtype=x.dtype, device="cuda") for x in (q, k, v))
    for at in _batches(state):
        rq, tq = _where(state["seg_q"], state["sizes_q"], at, hq)
        rk, tk = _where(seg_k, state["sizes_k"], at, hk)
        lq, lk = rq.shape[1], rk.shape[1]
        for h in [slice(0, hk)] if len(at) > 1 or rq.numel() * rk.numel() * hq <= PADDED else [slice(i, i + 1) for i in range(hk)]:
            hs, gs = h.stop - h.start, slice(h.start * (hq // hk), h.stop * (hq // hk))
            qs, ks, vs = _heads(q[:, gs], rq, tq, hs), _heads(k[:, h], rk, tk, hs), _heads(v[:, h], rk, tk, hs)
            do, o = _heads(state["do"][:, gs], rq, tq, hs), _heads(state["o"][:, gs], rq, tq, hs)
            lse = _heads(state["lse"][:, gs, None], rq, tq, hs)
            p = torch.exp(qs @ ks.transpose(2, 3) * scale - lse)
            p.masked_fill_(~tk[:, None, None, :], 0.0)
            delta = (do * o).sum(3, keepdim=True)
            ds = p * (do @ vs.transpose(2, 3) - delta) * scale
            here, there = rq[tq], rk[tk]
            dq[here, gs] = _rows_of(ds @ ks, len(at), hs, lq)[tq].to(dq.dtype)
            dk[there, h] = _rows_of(ds.transpose(2, 3) @ qs, len(at), hs, lk)[tk].to(dk.dtype)
            dv[there, h] = _rows_of(p.transpose(2, 3) @ do, len(at), hs, lk)[tk].to(dv.dtype)
    return {"dq": dq, "dk": dk, "dv": dv}


_PLAIN = {"norm": _plain_norm, "rope": _plain_rope, "route": _plain_route, "attn": _plain_attn}


# ------------------------------------------------------------- the library's way
def _library(state):
    import sparse_convolution_hash_gb300 as spc

    case = state["case"]
    op, back = case["op"], case["pass_"] == "bwd"
    if op == "norm":
        if not back:
            y, mean, rstd = spc.spc_layer_norm_fwd(state["x"], state["gamma"], state["beta"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dgamma, dbeta = spc.spc_layer_norm_bwd(state["dy"], state["x"], state["gamma"], state["mean"], state["rstd"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "rope":
        turn = spc.spc_rope_bwd if back else spc.spc_rope_fwd
        return turn(state["x"], state["coords"], state["steps"], _pairs(case))
    if op == "route":
        how = dict(score=spc.SPC_SCORE_SIGMOID if case["score"] == "sigmoid" else spc.SPC_SCORE_SOFTMAX,
                   renorm=case["renorm"], scale=case["scale"])
        if back:
            return spc.spc_route_bwd(state["dgate"], state["logits"], state["expert"], **how)
        expert, gate = spc.spc_route_fwd(state["logits"], case["k"], bias=state["bias"], groups=case["groups"],
                                         top_groups=case["kept"], **how)
        return {"expert": expert, "gate": gate}
    if not back:
        o, lse = spc.spc_attention_fwd(state["q"], state["k"], state["v"], state["seg_q"], seg_k=state["seg_k"])
        return {"o": o, "lse": lse}
    dq, dk, dv = spc.spc_attention_bwd(state["do"], state["q"], state["k"], state["v"], state["o"], state["lse"],
                                       state["seg_q"], seg_k=state["seg_k"])
    return {"dq": dq, "dk": dk, "dv": dv}


def run(state):
    return _library(state) if own else _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- floor work
def work(case):
    op, back, e = case["op"], case["pass_"] == "bwd", BYTES[case["type"]]
    if op == "norm":
        values = case["n"] * case["c"]
        return {"bytes": (3 if back else 2) * values * e + 8 * case["n"] + (12 if back else 8) * case["c"],
                "flops": (12 if back else 8) * values}
    if op == "rope":
        return {"bytes": 2 * case["n"] * case["heads"] * case["d"] * e + 16 * case["n"],
                "flops": 6 * case["n"] * case["heads"] * sum(_pairs(case))}
    if op == "route":
        n, experts, k = case["n"], case["experts"], case["k"]
        table = 4 * experts if case["bias"] and not back else 0
        return {"bytes": n * experts * e * (2 if back else 1) + 8 * n * k + table, "flops": 8 * n * experts}
    sizes_q, sizes_k = _attn_sizes(case)
    met = sum(a * b for a, b in zip(sizes_q, sizes_k))
    hq, hk, d = case["hq"], case["hk"], case["d"]
    rows = case["nq"] * hq * d * e, 2 * case["nk"] * hk * d * e
    moved = 4 * rows[0] + 2 * rows[1] if back else 2 * rows[0] + rows[1]
    return {"bytes": moved + 4 * case["nq"] * hq + 4 * (case["segments"] + 1) * (2 if case["cross"] else 1),
            "flops": (10 if back else 4) * met * hq * d}


# ------------------------------------------------------------------------- exact
def _exact_norm(case, s):
    x, gamma = s["x"].double(), s["gamma"].double()
    if case["pass_"] == "fwd":
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        return {"y": torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], gamma), "mean": mean, "rstd": rstd}
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    xh = (x - s["mean"].double()[:, None]) * rstd
    u, c = dy * gamma, case["c"]
    dx = (c * u - u.sum(1, keepdim=True) - xh * (u * xh).sum(1, keepdim=True)) * rstd / c
    return {"dx": dx, "dgamma": torch.einsum("nc,nc->c", dy, xh), "dbeta": torch.ones(len(x), dtype=x.dtype, device="cuda") @ dy}


def _exact_rope(case, s):
    out = s["x"].double().clone()
    at, sign = 0, -1.0 if case["pass_"] == "bwd" else 1.0
    for axis, count in enumerate(_pairs(case)):
        for j in range(count):
            turn = torch.polar(torch.ones(case["n"], dtype=torch.float64, device="cuda"),
                               sign * s["coords"][:, 1 + axis].double() * BASE ** (-j / count))
            z = torch.complex(out[:, :, 2 * at], out[:, :, 2 * at + 1]) * turn[:, None]
            out[:, :, 2 * at], out[:, :, 2 * at + 1] = z.real, z.imag
            at += 1
    return out


def _exact_route(case, s):
    logits = s["logits"].double()
    log_p = torch.nn.functional.logsigmoid(logits) if case["score"] == "sigmoid" else torch.log_softmax(logits, 1)
    if case["pass_"] == "bwd":
        z = logits.detach().requires_grad_()
        p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        gate = torch.gather(p, 1, s["expert"].long())
        gate = gate / gate.sum(1, keepdim=True) if case["renorm"] else gate
        return torch.autograd.grad((case["scale"] * gate * s["dgate"].double()).sum(), z)[0]
    expert = _plain_choice(s)[0]
    chosen = log_p.gather(1, expert)
    if case["renorm"]:
        chosen = chosen - torch.logsumexp(chosen, 1, keepdim=True)
    return {"expert": None, "gate": case["scale"] * torch.exp(chosen)}


def _exact_attn(case, s):
    q, k, v = (s[name].double() for name in ("q", "k", "v"))
    per, scale, back = case["hq"] // case["hk"], case["d"] ** -0.5, case["pass_"] == "bwd"
    if back:
        do, lse = s["do"].double(), s["lse"].double()
        delta = torch.einsum("nhd,nhd->nh", do, s["o"].double())
        out = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    else:
        out = {"o": torch.zeros_like(q), "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")}
    first_q = first_k = 0
    for nq, nk in zip(s["sizes_q"], s["sizes_k"]):
        keys = slice(first_k, first_k + nk)
        for at in range(first_q, first_q + nq if nk else first_q, 4096):
            rows = slice(at, min(at + 4096, first_q + nq))
            for h in range(case["hq"]):
                g = h // per
                z = torch.mm(q[rows, h], k[keys, g].T).mul_(scale)
                if not back:
                    out["lse"][rows, h] = torch.logsumexp(z, 1)
                    out["o"][rows, h] = torch.softmax(z, 1) @ v[keys, g]
                    continue
                p = torch.exp(z - lse[rows, h, None])
                ds = (torch.mm(do[rows, h], v[keys, g].T) - delta[rows, h, None]) * p * scale
                out["dv"][keys, g] += p.T @ do[rows, h]
                out["dk"][keys, g] += ds.T @ q[rows, h]
                out["dq"][rows, h] = ds @ k[keys, g]
        first_q, first_k = first_q + nq, first_k + nk
    return out


def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "route": _exact_route, "attn": _exact_attn}[case["op"]](case, s)
