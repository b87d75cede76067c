"""GPU parity of a transformer block's layers (layer norm, rotary positions, routing to experts, attention)
against plain float64 forms; the bounds come with them, from the arithmetic (block_ref.py)."""

import math

import numpy as np
import pytest
import torch

import block_ref as ref
import sparse_convolution_hash_gb300 as spc
from gpu_util import DT, dev

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std).to(DT[dtype])


def to(t):
    return None if t is None else t.to(dev())


def close(got, want, bound, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst by {float(((got - want).abs() / bound)[bad].max()):.3g} bounds"


# ------------------------------------------------------------------ layer norm
NORM = [(1, 1), (1, 16), (3, 8), (2000, 16), (513, 64), (77, 33), (300, 40), (129, 127), (65, 200), (1025, 96), (40, 260), (33, 512),
        (21, 520), (17, 1000), (50, 1024), (9, 1027), (7, 2048), (30, 384), (5, 4001), (12, 4096), (3, 9000), (4, 8192), (2, 20000), (0, 24),
        (40000, 24), (20000, 7)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,c", NORM)
def test_layer_norm(n, c, dtype):
    g = gen(n + c)
    x = normal(g, n, c, dtype="f32") * (0.5 + torch.rand(c, generator=g)) + normal(g, c)
    x = x.to(DT[dtype])
    ga, be = (1 + 0.3 * normal(g, c), 0.3 * normal(g, c)) if c % 2 == 0 else (None, None)
    dy = normal(g, n, c, dtype=dtype)
    want, bound = ref.layer_norm_fwd(x, ga, be, 1e-5)
    got = spc.spc_layer_norm_fwd(to(x), to(ga), to(be))
    for a, w, b, name in zip(got, want, bound, ("y", "mean", "rstd")):
        close(a, w, b, name)
    mean, rstd = got[1], got[2]
    want, bound = ref.layer_norm_bwd(dy, x, ga, mean.cpu(), rstd.cpu())
    back = spc.spc_layer_norm_bwd(to(dy), to(x), to(ga), mean, rstd)
    for a, w, b, name in zip(back, want, bound, ("dx", "dgamma", "dbeta")):
        close(a, w, b, name)
    again = spc.spc_layer_norm_bwd(to(dy), to(x), to(ga), mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(back, again))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", [33, 64, 600])
def test_layer_norm_in_place_far_means_and_odd_places(c, dtype):
    g = gen(c)
    x = (1000 + normal(g, 50, c)).to(DT[dtype])
    want, bound = ref.layer_norm_fwd(x, None, None, 1e-5)
    flat = torch.zeros(50 * c + 1, dtype=DT[dtype], device=dev())
    at = flat[1:].view(50, c)  # an element past a 16-byte boundary
    at.copy_(x)
    y, mean, rstd = spc.spc_layer_norm_fwd(at, None, None, out=at)
    assert y.data_ptr() == at.data_ptr() and flat[0] == 0
    for a, w, b in zip((y, mean, rstd), want, bound):
        close(a, w, b)
    dy = normal(g, 50, c, dtype=dtype)
    want, bound = ref.layer_norm_bwd(dy, x, None, mean.cpu(), rstd.cpu())
    at.copy_(dy)
    got = spc.spc_layer_norm_bwd(at, to(x), None, mean, rstd, out=at)
    for a, w, b in zip(got, want, bound):
        close(a, w, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,c,skip,skip_affine", [(37, 6, 0, 0), (70, 46, 2, 0), (19, 334, 0, 0), (19, 334, 2, 1), (19, 334, 0, 2), (11, 1002, 6, 0),
                                                  (5, 2050, 0, 0), (5, 4098, 2, 2), (3, 8186, 0, 0), (23, 333, 0, 0), (2, 9002, 2, 0), (64, 64, 2, 0)])
def test_layer_norm_in_words_of_two_and_one(n, c, skip, skip_affine, dtype):
    """Rows, gamma and beta off their 16-byte boundaries by a few elements."""
    g = gen(n + c + skip)

    def apart(t, by):
        flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=dev())
        flat[by:] = to(t).view(-1)
        return flat[by:].view(t.shape)

    x, dy = normal(g, n, c, dtype=dtype), normal(g, n, c, dtype=dtype)
    ga, be = 1 + 0.3 * normal(g, c), 0.3 * normal(g, c)
    want, bound = ref.layer_norm_fwd(x, ga, be, 1e-5)
    got = spc.spc_layer_norm_fwd(apart(x, skip), apart(ga, skip_affine), apart(be, skip_affine))
    for a, w, b, name in zip(got, want, bound, ("y", "mean", "rstd")):
        close(a, w, b, name)
    want, bound = ref.layer_norm_bwd(dy, x, ga, got[1].cpu(), got[2].cpu())
    back = spc.spc_layer_norm_bwd(apart(dy, skip), apart(x, skip), apart(ga, skip_affine), got[1], got[2])
    for a, w, b, name in zip(back, want, bound, ("dx", "dgamma", "dbeta")):
        close(a, w, b, name)


# ------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,heads,d,pairs,extra", [
    (1, 1, 2, (0, 0, 1), 0), (5, 3, 16, (2, 3, 3), 0), (300, 8, 64, (10, 11, 11), 4), (77, 5, 40, (6, 6, 6), 5), (33, 2, 7, (1, 1, 1), 1),
    (50, 1, 128, (0, 64, 0), 0), (9, 70, 24, (4, 4, 4), 0), (4000, 4, 96, (16, 16, 16), 2), (3, 2, 5, (0, 0, 0), 0), (0, 2, 8, (1, 1, 1), 0)])
def test_rope(n, heads, d, pairs, extra, dtype):
    g = gen(n + d)
    rows = normal(g, n, heads + extra, d, dtype=dtype)
    coords = torch.randint(0, 2000, (n, 4), generator=g, dtype=torch.int32)
    steps = spc.spc_rope_steps(pairs)
    x = to(rows)[:, :heads]
    for back, f in ((False, spc.spc_rope_fwd), (True, spc.spc_rope_bwd)):
        want, bound = ref.rope(rows[:, :heads], coords, pairs, 10000.0, back)
        close(f(x, to(coords), steps, pairs), want, bound)
        whole = to(rows)
        f(whole[:, :heads], to(coords), steps, pairs, out=whole[:, :heads])
        close(whole[:, :heads], want, bound)
        assert torch.equal(whole[:, heads:].cpu(), rows[:, heads:])


def test_rope_far_and_negative_cells():
    g = gen(7)
    pairs = (3, 2, 3)
    coords = torch.tensor([[0, -1, 2 ** 31 - 1, -2 ** 31], [0, 12345678, -87654321, 5], [1, 0, 0, 0]], dtype=torch.int32)
    x = normal(g, 3, 2, 16)
    want, bound = ref.rope(x, coords, pairs, 100.0)
    # float64's angle is off by 2^-53 of itself, the step by 2^-65 turns for each cell
    got = spc.spc_rope_fwd(to(x), to(coords), spc.spc_rope_steps(pairs, 100.0), pairs)
    close(got, want, bound + 2.0 ** -30)
    assert torch.equal(got[2].cpu(), x[2])
    x[0, 0, 0], x[1, 1, 2] = math.inf, math.nan  # stay in their pairs
    got = spc.spc_rope_fwd(to(x), to(coords), spc.spc_rope_steps((1, 1, 1), 100.0), (1, 1, 1))
    bad = ~got.isfinite().cpu()
    assert bad[0, 0, :2].all() and bad[1, 1, 2:4].all() and int(bad.sum()) == 4


# ----------------------------------------------------------- routing to experts
ROUTE = [  # n, experts, top_k, score, bias, groups, kept, renorm
    (1, 1, 1, "softmax", False, 1, 1, True), (300, 4, 3, "softmax", True, 4, 3, True), (290, 16, 5, "sigmoid", True, 2, 1, True),
    (150, 12, 2, "softmax", False, 3, 2, False), (77, 8, 8, "sigmoid", False, 1, 1, True), (5, 4, 4, "sigmoid", True, 1, 1, False), (70, 8, 2, "softmax", False, 1, 1, True),
    (65, 64, 6, "softmax", True, 1, 1, False), (33, 60, 4, "sigmoid", True, 4, 2, True), (129, 256, 8, "sigmoid", True, 8, 4, True),
    (40, 160, 3, "softmax", False, 4, 3, True), (17, 128, 8, "softmax", False, 1, 1, False), (9, 1000, 32, "sigmoid", False, 1, 1, True),
    (6, 1024, 5, "softmax", True, 512, 7, True), (31, 33, 3, "sigmoid", False, 11, 2, False), (21, 1024, 8, "sigmoid", True, 1024, 9, True)]


def route_case(n, experts, bias, dtype, seed=0):
    g = gen(seed + n + experts)
    logits = normal(g, n, experts, std=1.5).to(DT[dtype])
    return g, logits, normal(g, experts, std=0.1) if bias else None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,experts,top_k,score,bias,groups,kept,renorm", ROUTE)
def test_route(n, experts, top_k, score, bias, groups, kept, renorm, dtype):
    g, logits, b = route_case(n, experts, bias, dtype)
    kind = spc.SPC_SCORE_SIGMOID if score == "sigmoid" else spc.SPC_SCORE_SOFTMAX
    (expert, gate), bound = ref.route_fwd(logits, top_k, score, b, groups, kept, renorm, 2.5)
    got, w = spc.spc_route_fwd(to(logits), top_k, score=kind, bias=to(b), groups=groups, top_groups=kept, renorm=renorm, scale=2.5)
    assert torch.equal(got.cpu(), expert)
    close(w, gate, bound)
    dgate = normal(g, n, top_k)
    want, bound = ref.route_bwd(dgate, logits, expert, score, renorm, 2.5)
    st = spc.new_status(dev())
    close(spc.spc_route_bwd(to(dgate), to(logits), got, score=kind, renorm=renorm, scale=2.5, status=st), want, bound)
    spc.check_status(st)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_route_near_ties(score, groups, kept):
    """Scores that differ by less than fp32 shows: the choice is that of 64 bits."""
    g = gen(11)
    n, experts = 400, 32
    level = torch.randint(0, 4, (n, experts), generator=g)
    logits = (0.3 * level + 2.0 ** -22 * torch.randint(0, 3, (n, experts), generator=g)).float()
    bias = 2.0 ** -26 * torch.randint(0, 5, (experts,), generator=g).float() - 0.05 * torch.randint(0, 2, (experts,), generator=g)
    (expert, gate), bound = ref.route_fwd(logits, 5, score, bias, groups, kept, True, 1.0)
    kind = spc.SPC_SCORE_SIGMOID if score == "sigmoid" else spc.SPC_SCORE_SOFTMAX
    got, w = spc.spc_route_fwd(to(logits), 5, score=kind, bias=to(bias), groups=groups, top_groups=kept)
    assert torch.equal(got.cpu(), expert)
    close(w, gate, bound)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [True, False])
def test_route_masked_and_extreme_logits(score, renorm, biased):
    inf, nan = math.inf, math.nan
    rows = [[-inf] * 8, [nan] * 8, [-inf, nan, 1, -inf, nan, -inf, -inf, -inf], [inf, 1, inf, 0, -1, -inf, nan, 3],
            [-300, -301, -302, -500, -inf, -700, -650, -310], [3e38, -3e38, 0, 1, 2, 3, 4, 5], [0.0, -0.0] * 4, [-0.0, 0.0] * 4, [90, 100, 110, 88, -88, -90, 0, 1]]
    logits = torch.tensor(rows, dtype=torch.float32)
    bias = torch.linspace(0.5, -0.5, 8) if biased else None
    kind = spc.SPC_SCORE_SIGMOID if score == "sigmoid" else spc.SPC_SCORE_SOFTMAX
    (expert, gate), bound = ref.route_fwd(logits, 3, score, bias, 1, 1, renorm, 1.0)
    got, w = spc.spc_route_fwd(to(logits), 3, score=kind, bias=to(bias), renorm=renorm)
    assert torch.equal(got.cpu(), expert)
    close(w, gate, bound + 1e-30)
    dgate = torch.linspace(-1, 1, 27).view(9, 3)
    want, bound = ref.route_bwd(dgate, logits, expert, score, renorm, 1.0)
    close(spc.spc_route_bwd(to(dgate), to(logits), got, score=kind, renorm=renorm), want, bound + 1e-30)


@pytest.mark.parametrize("size", [2, 3, 8])
@pytest.mark.parametrize("best", [3e38, math.inf])
def test_route_groups_of_biases_at_the_end_of_fp32(size, best):
    """Sums of a group's two best that fp32 does not hold: groups are kept as their sums in 64 bits have it."""
    g = gen(12)
    logits = normal(g, 20, 5 * size)
    bias = torch.zeros(5 * size)
    for group, two in enumerate([(-3e38, -3e38), (-3e38, -2e38), (2.5e38, 3e38), (best, 3e38), (0.0, 0.0)]):
        bias[group * size:(group + 1) * size] = min(two)
        bias[(group + 1) * size - 1] = max(two)
    for kept in (1, 2, 4):
        k = min(2 * kept - 1, size * kept)
        (expert, gate), bound = ref.route_fwd(logits, k, "sigmoid", bias, 5, kept, True, 1.0)
        got, w = spc.spc_route_fwd(to(logits), k, score=spc.SPC_SCORE_SIGMOID, bias=to(bias), groups=5, top_groups=kept)
        assert torch.equal(got.cpu(), expert)
        close(w, gate, bound)


@pytest.mark.parametrize("size", [3, 4, 8])
def test_route_groups_whose_sums_cancel(size):
    """Biases of +-100 beside scores below 1: in fp32 a sum of two has lost the scores' last seven bits."""
    g = gen(13)
    n, groups = 400, 6
    experts = groups * size
    level = torch.randint(0, 3, (n, experts), generator=g)
    logits = (0.4 * level + 2.0 ** -18 * torch.randint(0, 5, (n, experts), generator=g)).float()
    bias = torch.full((groups, size), -100.0)
    bias[:, 0] = 100.0
    bias[:, 2:] = -200.0
    (expert, gate), bound = ref.route_fwd(logits, 3, "sigmoid", bias.view(-1), groups, 2, True, 1.0)
    got, w = spc.spc_route_fwd(to(logits), 3, score=spc.SPC_SCORE_SIGMOID, bias=to(bias.view(-1)), groups=groups, top_groups=2)
    assert torch.equal(got.cpu(), expert)
    close(w, gate, bound)


def test_route_reports_experts_out_of_range_and_feeds_row_segments():
    g, logits, _ = route_case(50, 16, False, "f32")
    expert, gate = spc.spc_route_fwd(to(logits), 2)
    seg, order = spc.spc_row_segments(expert.view(-1), 16)
    assert int(seg[-1]) == 100 and torch.equal(expert.view(-1)[order.long()].sort(stable=True).values, expert.view(-1)[order.long()])
    bad = expert.clone()
    bad[3, 1], bad[4, 0] = 16, -2
    st = spc.new_status(dev())
    spc.spc_route_bwd(gate, to(logits), bad, status=st)
    assert int(st.item()) == 10
    logits[7] = -math.inf
    logits[7, 3] = 1.0
    expert, gate = spc.spc_route_fwd(to(logits), 2)
    seg, _ = spc.spc_row_segments(expert.view(-1), 16)
    assert expert[7].tolist() == [3, -1] and gate[7].tolist() == [1.0, 0.0] and int(seg[-1]) == 99


# -------------------------------------------------------------------- attention
def offsets(sizes, before=0):
    return [before + sum(sizes[:i]) for i in range(len(sizes) + 1)]


ATTN = [  # hq, hk, d, query sizes, key sizes (None: the same), rows outside the segments
    (1, 1, 1, [1], None, 0), (2, 2, 16, [5], None, 0), (1, 1, 8, [64], None, 0), (2, 1, 64, [65, 1, 0, 130], None, 3),
    (4, 4, 32, [127, 129, 200], None, 0), (3, 3, 40, [300], None, 2), (4, 2, 128, [257, 100], None, 0), (6, 2, 72, [31, 97], None, 0),
    (8, 1, 64, [33, 3], [500, 129], 0), (2, 2, 64, [1, 1, 1], [700, 0, 333], 1), (4, 4, 24, [0, 40], [10, 90], 2),
    (2, 2, 7, [50, 20], None, 1), (1, 1, 100, [70], [130], 0), (5, 5, 33, [66], None, 0), (8, 8, 64, [513, 255], None, 0),
    (1, 1, 128, [1], [3000], 0), (16, 2, 128, [2, 1], [400, 900], 0), (2, 2, 80, [900], [40], 0), (2, 1, 16, [3] * 70, None, 5),
    (12, 4, 96, [140, 77], [260, 12], 0), (2, 2, 64, [1100], None, 0), (1, 1, 48, [0, 0], [0, 9], 0)]


def attn_case(hq, hk, d, sizes_q, sizes_k, outside, dtype, seed=0, std=1.5):
    g = gen(seed + d + sum(sizes_q))
    seg = offsets(sizes_q, outside)
    seg_k = seg if sizes_k is None else offsets(sizes_k, outside)
    nq, nk = seg[-1] + outside, seg_k[-1] + outside
    q, k, v = (normal(g, nq, hq, d, dtype=dtype, std=std), normal(g, nk, hk, d, dtype=dtype), normal(g, nk, hk, d, dtype=dtype))
    dout = normal(g, nq, hq, d, dtype=dtype)
    return q, k, v, dout, seg, seg_k


def on_cores(dtype, d):
    """Whether tensor cores take the call, and so probabilities are rounded."""
    return dtype != "f32" and d % 8 == 0


def run_attention(q, k, v, dout, seg, seg_k, dtype, scale=None, st=None):
    t_seg = torch.tensor(seg, dtype=torch.int32, device=dev())
    t_seg_k = None if seg_k is seg else torch.tensor(seg_k, dtype=torch.int32, device=dev())
    st = spc.new_status(dev()) if st is None else st
    o, lse = spc.spc_attention_fwd(to(q), to(k), to(v), t_seg, seg_k=t_seg_k, scale=scale, status=st)
    grads = spc.spc_attention_bwd(to(dout), to(q), to(k), to(v), o, lse, t_seg, seg_k=t_seg_k, scale=scale, status=st)
    spc.check_status(st)
    return o, lse, grads


def check_attention(q, k, v, dout, seg, seg_k, dtype, got, scale=None):
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, lse, grads = got
    (want, want_lse), (bound, bound_lse) = ref.attention_fwd(q, k, v, seg, seg_k, scale, on_cores(dtype, d))
    close(o, want, bound, "o")
    close(lse, want_lse, bound_lse, "lse")
    want, bound = ref.attention_bwd(dout, q, k, v, o.cpu(), lse.cpu(), seg, seg_k, scale, on_cores(dtype, d))
    for a, w, b, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        close(a, w, b, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hk,d,sizes_q,sizes_k,outside", ATTN)
def test_attention(hq, hk, d, sizes_q, sizes_k, outside, dtype):
    case = attn_case(hq, hk, d, sizes_q, sizes_k, outside, dtype)
    st = spc.new_status(dev())
    got = run_attention(*case, dtype, st=st)
    spc.check_status(st)
    check_attention(*case, dtype, got)
    again = run_attention(*case, dtype)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert all(torch.equal(a, b) for a, b in zip(got[2], again[2]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 40, 36])
def test_attention_on_slices_of_one_projection(d, dtype):
    g = gen(d)
    n, h, seg = 333, 3, [0, 200, 333]
    qkv, grad = normal(g, n, 3 * h, d, dtype=dtype), torch.full((n, 3 * h, d), 7.0, dtype=DT[dtype])
    q, k, v = qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:]
    dout = normal(g, n, h, d, dtype=dtype)
    t, dt, t_seg = to(qkv), to(grad), torch.tensor(seg, dtype=torch.int32, device=dev())
    parts = [t[:, i * h:(i + 1) * h] for i in range(3)]
    room = torch.full((n, 2 * h, d), 7.0, dtype=DT[dtype], device=dev())
    o, lse = spc.spc_attention_fwd(*parts, t_seg, out=room[:, :h])
    assert bool((room[:, h:] == 7).all())
    grads = spc.spc_attention_bwd(to(dout), *parts, o, lse, t_seg, dq=dt[:, :h], dk=dt[:, h:2 * h], dv=dt[:, 2 * h:])
    check_attention(q, k, v, dout, seg, seg, dtype, (o, lse, grads))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sizes_q,sizes_k", [([70, 130, 9], None), ([2, 2, 1], [70, 1000, 300]), ([1000, 20, 7], [3, 20, 70])])
def test_attention_segments_do_not_meet(sizes_q, sizes_k, dtype):
    """NaN and infinities of one segment's rows, and of rows of no segment, stay there."""
    q, k, v, dout, seg, seg_k = attn_case(2, 2, 64, sizes_q, sizes_k, 4, dtype)
    clean = run_attention(q, k, v, dout, seg, seg_k, dtype)
    a, b = slice(seg[1], seg[2]), slice(seg_k[1], seg_k[2])
    for t, rows in ((q, a), (dout, a), (k, b), (v, b)):
        t[rows] = math.nan
        t[:4], t[-4:] = math.inf, math.nan
    o, lse, grads = run_attention(q, k, v, dout, seg, seg_k, dtype)
    for got, want, rows in zip((o, lse, *grads), (clean[0], clean[1], *clean[2]), (a, a, a, b, b)):
        keep = torch.ones(got.shape[0], dtype=torch.bool, device=dev())
        keep[rows] = False
        assert torch.equal(got[keep], want[keep])
        assert bool(got[rows].isnan().any())
    assert bool((o[:4] == 0).all()) and bool((lse[-4:] == -math.inf).all()) and all(bool((x[-4:] == 0).all()) for x in grads)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("std", [0.0, 12.0, 60.0])
def test_attention_of_flat_and_peaked_scores(std, dtype):
    case = attn_case(2, 1, 64, [300, 140], None, 0, dtype, std=std)
    check_attention(*case, dtype, run_attention(*case, dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_of_growing_scores(dtype):
    """Each tile of keys holds a larger score than the ones before it, so the running maximum moves every time."""
    q, k, v, dout, seg, seg_k = attn_case(1, 1, 32, [700], None, 0, dtype)
    k = (k.float() * 0.05 + torch.linspace(0, 3, 700)[:, None, None]).to(DT[dtype])
    q = (q.float() * 0.05 + 1).to(DT[dtype])
    case = q, k, v, dout, seg, seg_k
    check_attention(*case, dtype, run_attention(*case, dtype, 1.0), 1.0)


@pytest.mark.parametrize("size", [1e-4, 300.0])
def test_attention_gradients_in_fp16_keep_their_digits(size):
    """Small and large gradients: ds has its own scale."""
    q, k, v, dout, seg, seg_k = attn_case(2, 2, 64, [900], None, 0, "f16")
    case = q, k, v, (dout.double() * size).half(), seg, seg_k
    o, lse, grads = run_attention(*case, "f16")
    want, bound = ref.attention_bwd(case[3], q, k, v, o.cpu(), lse.cpu(), seg, seg_k, 64 ** -0.5, True)
    for a, w, b in zip(grads, want, bound):
        close(a, w, b)


def test_attention_scores_of_minus_infinity():
    """A key that no query may see, and a query that sees none."""
    for dtype in TYPES:
        q, k, v, dout, seg, _ = attn_case(1, 1, 16, [200], None, 0, dtype)
        q, k = q.abs() + 0.1, k.clone()
        k[130:] = -math.inf
        o, lse = spc.spc_attention_fwd(to(q), to(k), to(v), torch.tensor(seg, dtype=torch.int32, device=dev()))
        (want, want_lse), (bound, bound_lse) = ref.attention_fwd(q, k[:130], v[:130], [0, 200], [0, 130], 0.25, dtype != "f32")
        close(o, want, bound)
        close(lse, want_lse, bound_lse)
        k[:] = -math.inf
        o, lse = spc.spc_attention_fwd(to(q), to(k), to(v), torch.tensor(seg, dtype=torch.int32, device=dev()))
        assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_without_rows(dtype):
    z = torch.zeros(0, 2, 16, dtype=DT[dtype], device=dev())
    x = torch.randn(5, 2, 16, device=dev()).to(DT[dtype])
    none, five = (torch.tensor(s, dtype=torch.int32, device=dev()) for s in ([0, 0], [0, 5]))
    o, lse = spc.spc_attention_fwd(x, z, z, five, seg_k=none)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv = spc.spc_attention_bwd(x, x, z, z, o, lse, five, seg_k=none)
    assert bool((dq == 0).all()) and dk.shape == z.shape
    o, lse = spc.spc_attention_fwd(z, x, x, none, seg_k=five)
    assert o.shape == z.shape and lse.shape == (0, 2)
    dq, dk, dv = spc.spc_attention_bwd(z, z, x, x, o, lse, none, seg_k=five)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.parametrize("seg", [[0, 40, 20, 60], [-5, 10, 20, 60], [0, 10, 20, 70]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_reports_bad_offsets(seg, dtype):
    x = torch.randn(60, 2, 32, device=dev()).to(DT[dtype])
    st = spc.new_status(dev())
    t = torch.tensor(seg, dtype=torch.int32, device=dev())
    o, lse = spc.spc_attention_fwd(x, x, x, t, status=st)
    assert int(st.item()) == 10
    st.zero_()
    spc.spc_attention_bwd(x, x, x, x, o, lse, t, status=st)
    assert int(st.item()) == 10


def test_attention_many_small_segments():
    """More segments than a warp searches in two turns."""
    g = np.random.default_rng(5)
    sizes = g.integers(0, 6, 1500).tolist()
    case = attn_case(2, 2, 32, sizes, None, 3, "bf16")
    check_attention(*case, "bf16", run_attention(*case, "bf16"))


def test_calls_in_a_graph_on_another_stream():
    """Captured once, replayed on new inputs."""
    g = gen(9)
    n, h, d, pairs = 300, 2, 64, (10, 11, 11)
    seg = torch.tensor([0, 120, 300], dtype=torch.int32, device=dev())
    coords = torch.randint(0, 100, (n, 4), generator=g, dtype=torch.int32).to(dev())
    steps = spc.spc_rope_steps(pairs)
    x = normal(g, n, 3 * h * d, dtype="bf16").to(dev())
    logits = normal(g, n, 16).to(dev())

    def block(x, logits):
        y, mean, rstd = spc.spc_layer_norm_fwd(x, None, None)
        qkv = y.view(n, 3 * h, d)
        turned = spc.spc_rope_fwd(qkv[:, :2 * h], coords, steps, pairs)
        o, lse = spc.spc_attention_fwd(turned[:, :h], turned[:, h:], qkv[:, 2 * h:], seg)
        grads = spc.spc_attention_bwd(o, turned[:, :h], turned[:, h:], qkv[:, 2 * h:], o, lse, seg)
        expert, gate = spc.spc_route_fwd(logits, 2)
        dl = spc.spc_route_bwd(gate, logits, expert)
        dx = spc.spc_layer_norm_bwd(x, x, None, mean, rstd)
        return [o, lse, *grads, expert, gate, dl, *dx]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block(x, logits)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = block(x, logits)
    torch.cuda.current_stream().wait_stream(stream)
    x.copy_(normal(g, n, 3 * h * d, dtype="bf16"))
    logits.copy_(normal(g, n, 16))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, block(x, logits)):
        assert torch.equal(a, b)
