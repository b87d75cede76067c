"""The learned block around the sparse convolutions, one operator at a time.

Rows of a batch lie in one [n, C] matrix, each row a voxel.  A segment is the
rows of one sample or of one expert: `seg` [S + 1] holds the offsets of the
segments among the rows in grouped order, and `order` [n] the row that stands at
each position (absent: the rows lie in that order already).

  segments  rows grouped by a small key: offsets and a stable order
  norm      group norm per sample with an activation, forward and backward
  dropout   dropout from a counter-based generator, with an added residual
  experts   products of each row with the weight of its expert: forward,
            gradient by the input, gradient by the weights

`listed()` and `draw()` give cases, `prepare()` a case's inputs, `run()` one
pass: the plain form in 32 bits, or the library's kernels where `own` is true.
`work()` counts what a pass has to move and compute; `exact()` is the definition
in 64 bits.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one sample of the 32^3 set: the smallest call, where latency counts
        dict(name="norm_fwd_2k_f32", op="norm", pass_="fwd", n=2000, c=16, groups=4, samples=1,
             act="silu", type="f32", shuffled=False),
        # the 4 x 192^3 shells of the training step, sorted rows
        dict(name="norm_fwd_shells_bf16", op="norm", pass_="fwd", n=498145, c=64, groups=32,
             samples=4, act="silu", type="bf16", shuffled=False),
        dict(name="norm_bwd_shells_bf16", op="norm", pass_="bwd", n=498145, c=64, groups=32,
             samples=4, act="silu", type="bf16", shuffled=False),
        # an odd number of rows and of groups, samples of very unequal size, rows in no order
        dict(name="norm_bwd_ragged_f16", op="norm", pass_="bwd", n=33333, c=40, groups=5,
             samples=7, act="silu", type="f16", shuffled=True),
        # the end of a residual block on the 256^3 shell
        dict(name="dropout_fwd_shell_bf16", op="dropout", pass_="fwd", n=398833, c=128, p=0.1,
             residual=True, type="bf16"),
        # the gradient of a narrow head: an odd number of values
        dict(name="dropout_bwd_odd_f16", op="dropout", pass_="bwd", n=12345, c=33, p=0.5,
             residual=False, type="f16"),
        # the sample of each voxel of a LiDAR batch, read from the coordinates' first column
        dict(name="segments_lidar", op="segments", n=120000, segments=2, column=True, dropped=0.0),
        # the experts of 65,536 tokens, two each
        dict(name="segments_route", op="segments", n=131072, segments=64, column=False, dropped=0.0),
        # the first product of a feed-forward layer of 16 experts
        dict(name="experts_fwd_bf16", op="experts", pass_="fwd", m=32768, cin=1024, cout=4096,
             experts=16, slots=1, type="bf16", dropped=0.0),
        # its gradient in a narrower layer: two experts to a token, some slots without one
        dict(name="experts_dgrad_f16", op="experts", pass_="dgrad", m=49998, cin=256, cout=1024,
             experts=64, slots=2, type="f16", dropped=0.03),
        dict(name="experts_wgrad_bf16", op="experts", pass_="wgrad", m=32768, cin=512, cout=2048,
             experts=8, slots=1, type="bf16", dropped=0.0),
        # sixteen tokens, two experts to each: the weights are read and little else
        dict(name="experts_few_bf16", op="experts", pass_="fwd", m=32, cin=1024, cout=4096,
             experts=64, slots=2, type="bf16", dropped=0.0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["segments", "norm", "norm", "dropout", "experts", "experts"])
    if op == "segments":
        return dict(op=op, n=_spread(rng, 1000, 1000000), segments=_spread(rng, 1, 256),
                    column=rng.random() < 0.5, dropped=rng.choice([0.0, 0.05]))
    type_ = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "norm":
        per = rng.choice([1, 2, 4, 5, 8, 16])
        groups = rng.choice([1, 4, 8, 13, 32])
        return dict(op=op, pass_=rng.choice(["fwd", "bwd"]), n=_spread(rng, 500, 32000000 // (256 + per * groups)),
                    c=per * groups, groups=groups, samples=rng.choice([1, 2, 3, 8, 21]),
                    act=rng.choice(["none", "silu", "silu"]), type=type_, shuffled=rng.random() < 0.4)
    if op == "dropout":
        c = _spread(rng, 8, 512)
        return dict(op=op, pass_=rng.choice(["fwd", "bwd"]), n=_spread(rng, 100, 48000000 // c), c=c,
                    p=rng.choice([0.05, 0.1, 0.3, 0.5]), residual=rng.random() < 0.5, type=type_)
    slots = rng.choice([1, 2])
    tokens = _spread(rng, 1, 16000)
    cin = rng.choice([64, 100, 128, 200, 256, 512, 1024])
    cout = rng.choice([64, 128, 136, 256, 512, 1000, 2048])
    if type_ == "f32":
        tokens = min(tokens, 4000)
    return dict(op=op, pass_=rng.choice(["fwd", "dgrad", "wgrad"]), m=tokens * slots, cin=cin, cout=cout,
                experts=rng.choice([2, 5, 8, 16, 64]), slots=slots, type=type_,
                dropped=rng.choice([0.0, 0.0, 0.05]))


# ----------------------------------------------------------------------- inputs
def _keys(n, segments, skew, dropped, gen):
    """A key for each row: segments of unequal popularity, some rows without one (-1)."""
    weight = torch.exp(skew * torch.randn(segments, generator=gen, device="cuda"))
    edges = torch.cumsum(weight / weight.sum(), 0)
    ids = torch.searchsorted(edges, torch.rand(n, generator=gen, device="cuda")).clamp_(max=segments - 1)
    if dropped > 0:
        ids = torch.where(torch.rand(n, generator=gen, device="cuda") < dropped, -1, ids)
    return ids.to(torch.int32)


def _grouped(ids, segments):
    """Offsets and stable order of the keys, with the sizes a program knows on the host."""
    key = torch.where((ids < 0) | (ids >= segments), segments, ids.long())
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=segments + 1)[:segments]
    seg = torch.zeros(segments + 1, dtype=torch.int32, device="cuda")
    seg[1:] = torch.cumsum(counts, 0)
    return seg, order.to(torch.int32), counts.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, type_=None):
        a = torch.randn(*shape, generator=gen, device="cuda") * std
        return a.to(TYPES[type_ or case["type"]])

    if op == "segments":
        ids = _keys(case["n"], case["segments"], 0.5, case["dropped"], gen)
        if case["column"]:
            coords = torch.randint(0, 1024, (case["n"], 4), generator=gen, device="cuda", dtype=torch.int32)
            coords[:, 0] = ids
            ids = coords[:, 0]
        return dict(case=case, ids=ids)
    if op == "norm":
        n, c = case["n"], case["c"]
        ids = _keys(n, case["samples"], 0.5, 0.0, gen)
        if not case["shuffled"]:
            ids = torch.sort(ids).values
        seg, order, sizes = _grouped(ids, case["samples"])
        # features of a convolution: every channel with a mean and a spread of its own
        x = torch.randn(n, c, generator=gen, device="cuda")
        x = x * torch.empty(c, device="cuda").uniform_(0.5, 2.0, generator=gen) + normal(c, type_="f32")
        state = dict(case=case, x=x.to(TYPES[case["type"]]), gamma=1 + normal(c, std=0.2, type_="f32"),
                     beta=normal(c, std=0.2, type_="f32"), seg=seg, order=order if case["shuffled"] else None,
                     longest=max(sizes))
        if case["pass_"] == "bwd":
            state["dy"] = normal(n, c)
            mean, rstd = _plain_stats(state)
            state["mean"], state["rstd"] = mean, rstd
        return state
    if op == "dropout":
        shape = (case["n"], case["c"])
        rng = torch.randint(0, 2 ** 62, (2,), generator=gen, device="cuda", dtype=torch.int64)
        return dict(case=case, x=normal(*shape), residual=normal(*shape) if case["residual"] else None, rng=rng)
    m, slots = case["m"], case["slots"]
    cin, cout, experts = case["cin"], case["cout"], case["experts"]
    seg, order, sizes = _grouped(_keys(m, experts, 0.4, case["dropped"], gen), experts)
    state = dict(case=case, seg=seg, longest=max(max(sizes), 1),
                 used=torch.tensor([g for g in range(experts) if sizes[g]] or [0], dtype=torch.int64, device="cuda"))
    if case["pass_"] != "wgrad":
        state["w"] = normal(experts, cin, cout, std=1.0 / math.sqrt(cin if case["pass_"] == "fwd" else cout))
    # a token's slots are neighbours, and each slot is a row of the result; with
    # one slot the rows were brought into grouped order before
    if slots > 1:
        state["x_rows"] = order // slots if case["pass_"] != "dgrad" else order
        state["y_rows"] = order
    else:
        state["x_rows"] = state["y_rows"] = None
    if case["pass_"] != "dgrad":
        state["x"] = normal(m // slots, cin)
    if case["pass_"] != "fwd":
        state["dy"] = normal(m, cout)
    return state


# ------------------------------------------------------------------ plain forms
def _padded(state):
    """Positions of each segment side by side [S, longest], which of them there are, and each position's segment."""
    seg = state["seg"].long()
    step = torch.arange(state["longest"], device="cuda")
    there = step < (seg[1:] - seg[:-1])[:, None]
    return torch.where(there, seg[:-1, None] + step, 0), there


def _segment_of(state, n):
    """The segment of each position (S past the last one)."""
    return torch.searchsorted(state["seg"][1:].contiguous(), torch.arange(n, device="cuda", dtype=torch.int32), right=True)


def _sums(values, state, rows, there):
    """Sums over each segment and each group of channels: [S, G]."""
    s, length = there.shape
    picked = torch.where(there[:, :, None], values[rows], 0.0)
    return picked.sum(1).view(s, state["case"]["groups"], -1).sum(2)


def _rows(state):
    at, there = _padded(state)
    return (at if state["order"] is None else state["order"].long()[at]), there


def _by_row(state, table):
    """A row's entry of a table [S, G], once for each of its channels: [n, C]."""
    n, c = state["x"].shape
    of = _segment_of(state, n)
    if state["order"] is not None:
        of = torch.empty_like(of).scatter_(0, state["order"].long(), of)
    return table.repeat_interleave(c // state["case"]["groups"], 1)[of]


def _plain_stats(state):
    case = state["case"]
    rows, there = _rows(state)
    x = state["x"].float()
    count = (there.sum(1, keepdim=True) * (case["c"] // case["groups"])).clamp(min=1)
    mean = _sums(x, state, rows, there) / count
    var = _sums((x - _by_row(state, mean)) ** 2, state, rows, there) / count
    return mean, 1.0 / torch.sqrt(var + EPS)


def _plain_norm_fwd(state):
    mean, rstd = _plain_stats(state)
    z = (state["x"].float() - _by_row(state, mean)) * _by_row(state, rstd) * state["gamma"] + state["beta"]
    y = z / (1 + torch.exp(-z)) if state["case"]["act"] == "silu" else z
    return {"y": y.to(state["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(state):
    case = state["case"]
    gamma, beta = state["gamma"], state["beta"]
    rstd = _by_row(state, state["rstd"])
    xh = (state["x"].float() - _by_row(state, state["mean"])) * rstd
    dz = state["dy"].float()
    if case["act"] == "silu":
        z = xh * gamma + beta
        sig = 1 / (1 + torch.exp(-z))
        dz = dz * sig * (1 + z * (1 - sig))
    rows, there = _rows(state)
    count = (there.sum(1, keepdim=True) * (case["c"] // case["groups"])).clamp(min=1)
    a = _sums(dz * gamma, state, rows, there) / count
    b = _sums(dz * gamma * xh, state, rows, there) / count
    dx = rstd * (dz * gamma - _by_row(state, a) - xh * _by_row(state, b))
    return {"dx": dx.to(state["x"].dtype), "dgamma": (dz * xh).sum(0), "dbeta": dz.sum(0)}


def _mul32(a, b):
    """High and low halves of the product of 32-bit words held in 64-bit ones."""
    low, high = a * (b & 0xFFFF), a * (b >> 16)
    mid = high + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _words(rng, n):
    """The first n words of the counter-based generator (Philox, 4 words of 32 bits, 10 rounds)."""
    quad = torch.arange((n + 3) // 4, device="cuda")
    k0, k1 = rng[0] & 0xFFFFFFFF, (rng[0] >> 32) & 0xFFFFFFFF
    c0, c1 = quad & 0xFFFFFFFF, quad >> 32
    c2, c3 = (rng[1] & 0xFFFFFFFF).expand_as(quad), ((rng[1] >> 32) & 0xFFFFFFFF).expand_as(quad)
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack([c0, c1, c2, c3], 1).view(-1)[:n]


def _plain_dropout(state):
    x, p = state["x"], state["case"]["p"]
    keep = _words(state["rng"], x.numel()).view(x.shape) >= round(p * 2 ** 32)
    y = torch.where(keep, x.float() * (1 / (1 - p)), 0.0)
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(x.dtype)


def _plain_segments(state):
    ids, segments = state["ids"], state["case"]["segments"]
    key = torch.where((ids < 0) | (ids >= segments), segments, ids)
    seg = (key[:, None] < torch.arange(segments + 1, device="cuda", dtype=torch.int32)).sum(0) if segments <= 4 else \
        torch.zeros(segments + 2, dtype=torch.int64, device="cuda").index_add_(0, key.long() + 1, torch.ones_like(key, dtype=torch.int64)).cumsum(0)[:-1]
    return {"seg": seg.to(torch.int32), "order": torch.argsort(key, stable=True).to(torch.int32)}


def _spots(state, m):
    """Where the row at each position stands in the padded layout of the used experts, and whether it has an expert."""
    of = _segment_of(state, m)
    there = of < state["case"]["experts"]
    of = torch.where(there, of, 0)
    place = torch.searchsorted(state["used"], of).clamp(max=state["used"].numel() - 1)
    return place * state["longest"] + torch.arange(m, device="cuda") - state["seg"].long()[of], there[:, None]


def _picked(values, rows, at, there):
    at = at if rows is None else rows.long()[at]
    return torch.where(there[:, :, None], values[at].float(), 0.0)


def _plain_experts(state):
    case, used = state["case"], state["used"]
    m, pass_ = case["m"], case["pass_"]
    at, there = _padded(state)
    at, there = at[used], there[used]
    if pass_ == "wgrad":
        dw = torch.zeros(case["experts"], case["cin"], case["cout"], device="cuda")
        dw[used] = torch.bmm(_picked(state["x"], state["x_rows"], at, there).transpose(1, 2),
                             _picked(state["dy"], state["y_rows"], at, there))
        return dw
    w = state["w"][used].float()
    if pass_ == "fwd":
        got, to = torch.bmm(_picked(state["x"], state["x_rows"], at, there), w), state["y_rows"]
    else:
        got, to = torch.bmm(_picked(state["dy"], state["y_rows"], at, there), w.transpose(1, 2)), state["x_rows"]
    spot, has = _spots(state, m)
    got = torch.where(has, got.view(-1, got.shape[2])[spot.clamp(max=got.shape[0] * got.shape[1] - 1)], 0.0).to(state["w"].dtype)
    return got if to is None else torch.empty_like(got).index_copy_(0, to.long(), got)


def _plain(state):
    case = state["case"]
    if case["op"] == "segments":
        return _plain_segments(state)
    if case["op"] == "norm":
        return _plain_norm_fwd(state) if case["pass_"] == "fwd" else _plain_norm_bwd(state)
    if case["op"] == "dropout":
        return _plain_dropout(state)
    return _plain_experts(state)


# ------------------------------------------------------------- the library's way
def _library(state):
    import sparse_convolution_hash_gb300 as spc

    case = state["case"]
    if case["op"] == "segments":
        seg, order = spc.spc_row_segments(state["ids"], case["segments"])
        return {"seg": seg, "order": order}
    if case["op"] == "dropout":
        if case["pass_"] == "bwd" and state["residual"] is None:
            return spc.spc_dropout_bwd(state["x"], case["p"], state["rng"])
        return spc.spc_dropout_fwd(state["x"], case["p"], state["rng"], residual=state["residual"])
    if case["op"] == "norm":
        act = spc.SPC_ACT_SILU if case["act"] == "silu" else spc.SPC_ACT_NONE
        if case["pass_"] == "fwd":
            y, mean, rstd = spc.spc_group_norm_fwd(state["x"], state["gamma"], state["beta"], state["seg"],
                                                   case["groups"], order=state["order"], eps=EPS, act=act)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dgamma, dbeta = spc.spc_group_norm_bwd(state["dy"], state["x"], state["gamma"], state["beta"],
                                                   state["mean"], state["rstd"], state["seg"], case["groups"],
                                                   order=state["order"], act=act)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    rows = dict(x_rows=state["x_rows"], y_rows=state["y_rows"])
    if case["pass_"] == "fwd":
        return spc.spc_grouped_fwd(state["x"], state["w"], state["seg"], **rows)
    if case["pass_"] == "dgrad":
        return spc.spc_grouped_dgrad(state["dy"], state["w"], state["seg"], **rows)
    return spc.spc_grouped_wgrad(state["x"], state["dy"], state["seg"], **rows)


def run(state):
    return _library(state) if own else _plain(state)


# -------------------------------------------------------------------- floor work
def work(case):
    op = case["op"]
    if op == "segments":
        return {"bytes": 8 * case["n"] + 4 * (case["segments"] + 1), "flops": 0}
    e = BYTES[case["type"]]
    if op == "norm":
        values, back = case["n"] * case["c"], case["pass_"] == "bwd"
        table = 8 * case["c"] * (2 if back else 1) + 8 * case["samples"] * case["groups"] + 4 * (case["samples"] + 1)
        rows = 4 * case["n"] if case["shuffled"] else 0
        return {"bytes": (3 if back else 2) * values * e + table + rows, "flops": (25 if back else 12) * values}
    if op == "dropout":
        values = case["n"] * case["c"]
        return {"bytes": (3 if case["residual"] else 2) * values * e, "flops": 3 * values}
    m, cin, cout, experts, slots = case["m"], case["cin"], case["cout"], case["experts"], case["slots"]
    routed = m * (1 - case["dropped"])
    touched = experts * (1 - (1 - 1 / experts) ** routed)
    lists = (8 if slots > 1 else 0) * m + 4 * (experts + 1)
    if case["pass_"] == "wgrad":
        moved = m // slots * cin * e + m * cout * e + experts * cin * cout * 4
    elif case["pass_"] == "fwd":
        moved = m // slots * cin * e + m * cout * e + touched * cin * cout * e
    else:
        moved = m * cin * e + m * cout * e + touched * cin * cout * e
    return {"bytes": moved + lists, "flops": 2 * routed * cin * cout}


# ------------------------------------------------------------------------- exact
def _bounds(state):
    seg = state["seg"].tolist()
    return list(zip(seg[:-1], seg[1:]))


def _at(rows, lo, hi):
    return slice(lo, hi) if rows is None else rows[lo:hi].long()


def _exact_norm(case, s):
    x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
    n, c = x.shape
    groups, per = case["groups"], c // case["groups"]
    means, rstds = [], []
    first, dgamma, dbeta = torch.zeros_like(x), torch.zeros_like(gamma), torch.zeros_like(beta)
    for k, (lo, hi) in enumerate(_bounds(s)):
        at = _at(s["order"], lo, hi)
        v = x[at].view(hi - lo, groups, per)
        if case["pass_"] == "fwd":
            mean = v.mean((0, 2)) if hi > lo else torch.zeros(groups, dtype=x.dtype, device=x.device)
            var = v.var((0, 2), unbiased=False) if hi > lo else torch.zeros_like(mean)
            rstd = (var + EPS) ** -0.5
            means.append(mean)
            rstds.append(rstd)
        else:
            mean, rstd = s["mean"][k].double(), s["rstd"][k].double()
        xh = (v - mean[:, None]) * rstd[:, None]
        z = xh.reshape(hi - lo, c) * gamma + beta
        sig = torch.sigmoid(z)
        if case["pass_"] == "fwd":
            first[at] = z * sig if case["act"] == "silu" else z
            continue
        dz = s["dy"][at].double()
        if case["act"] == "silu":
            dz = dz * (sig + z * sig * (1 - sig))
        xh = xh.reshape(hi - lo, c)
        dgamma += (dz * xh).sum(0)
        dbeta += dz.sum(0)
        if hi == lo:
            continue
        u, w = (dz * gamma).view(-1, groups, per), xh.view(-1, groups, per)
        first[at] = ((u - u.mean((0, 2))[:, None] - w * (u * w).mean((0, 2))[:, None]) * rstd[:, None]).reshape(-1, c)
    if case["pass_"] == "fwd":
        return {"y": first, "mean": torch.stack(means), "rstd": torch.stack(rstds)}
    return {"dx": first, "dgamma": dgamma, "dbeta": dbeta}


def _exact_words(seed, offset, n):
    """The generator by its published rounds, in numpy's wrapping 64-bit words."""
    u = np.uint64
    word, m0, m1 = u(0xFFFFFFFF), u(0xD2511F53), u(0xCD9E8D57)
    quads = np.arange((n + 3) // 4, dtype=u)
    c = [quads & word, quads >> u(32), np.full_like(quads, offset & 0xFFFFFFFF), np.full_like(quads, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = m0 * c[0], m1 * c[2]
        c = [(q >> u(32)) ^ c[1] ^ u(key[0]), q & word, (p >> u(32)) ^ c[3] ^ u(key[1]), p & word]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, 1).reshape(-1)[:n]


def _exact_dropout(case, s):
    words = _exact_words(int(s["rng"][0]), int(s["rng"][1]), s["x"].numel())
    keep = torch.from_numpy(words >= np.uint64(round(case["p"] * 2 ** 32))).to("cuda").view(s["x"].shape)
    y = torch.where(keep, s["x"].double() / (1 - case["p"]), 0.0)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_experts(case, s):
    x_rows, y_rows = s["x_rows"], s["y_rows"]
    if case["pass_"] == "wgrad":
        out = torch.zeros(case["experts"], case["cin"], case["cout"], dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(case["m"], case["cout" if case["pass_"] == "fwd" else "cin"], dtype=torch.float64, device="cuda")
    for g, (lo, hi) in enumerate(_bounds(s)):
        if hi == lo:
            continue
        xa, ya = _at(x_rows, lo, hi), _at(y_rows, lo, hi)
        if case["pass_"] == "fwd":
            out[ya] = s["x"][xa].double() @ s["w"][g].double()
        elif case["pass_"] == "dgrad":
            out[xa] = s["dy"][ya].double() @ s["w"][g].double().T
        else:
            out[g] = s["x"][xa].double().T @ s["dy"][ya].double()
    return out


def exact(case, seed):
    if case["op"] == "segments":
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return _exact_dropout(case, s) if case["op"] == "dropout" else _exact_experts(case, s)
