"""A transformer block's layers in the corners of their ranges.

Bounds are those of block_ref.py, or derived beside the test from the same arithmetic (E = 2^-24)."""

import math

import pytest
import torch

import block_ref as ref
import sparse_convolution_hash_gb300 as spc
from block_ref import E
from gpu_util import DT, dev
from test_gpu_block import TYPES, close, gen, normal, to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def offsets(*seg):
    return torch.tensor(seg, dtype=torch.int32, device=dev())


# ------------------------------------------------------------------ no rows on one side
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hk", [(8, 8), (8, 2)])
@pytest.mark.parametrize("n", [1000, 20000])
def test_attention_gradients_where_one_side_has_no_rows(n, hq, hk, dtype):
    """Many rows on the other side, whose walk would be split."""
    q, k = (normal(gen(n), n, h, 16, dtype=dtype).to(dev()) for h in (hq, hk))
    none_q, none_k = q[:0], k[:0]
    no, all_ = offsets(0, 0), offsets(0, n)
    o, lse = spc.spc_attention_fwd(q, none_k, none_k, all_, seg_k=no)
    assert not o.any() and bool((lse == -math.inf).all())
    dq, dk, dv = spc.spc_attention_bwd(q, q, none_k, none_k, o, lse, all_, seg_k=no, dq=torch.full_like(q, 7))
    assert not dq.any() and dk.shape == dv.shape == none_k.shape
    o, lse = spc.spc_attention_fwd(none_q, k, k, no, seg_k=all_)
    dq, dk, dv = spc.spc_attention_bwd(none_q, none_q, k, k, o, lse, no, seg_k=all_, dk=torch.full_like(k, 7), dv=torch.full_like(k, 7))
    assert dq.shape == none_q.shape and not dk.any() and not dv.any()


# ------------------------------------------------------------------ ties at the border of a choice
def check_choice(logits, top_k, score, bias, groups=1, kept=1):
    (expert, gate), bound = ref.route_fwd(logits, top_k, score, bias, groups, kept, True, 1.0)
    kind = spc.SPC_SCORE_SIGMOID if score == "sigmoid" else spc.SPC_SCORE_SOFTMAX
    got, w = spc.spc_route_fwd(to(logits), top_k, score=kind, bias=to(bias), groups=groups, top_groups=kept)
    wrong = (got.cpu() != expert).any(1).nonzero()[:, 0]
    assert not len(wrong), f"{len(wrong)} rows, the first {int(wrong[0])}: {got[wrong[0]].tolist()}, not {expert[wrong[0]].tolist()}"
    close(w, gate, bound)


@pytest.mark.parametrize("score,low,high,dtype", [
    ("sigmoid", 15.5, 16.0, "f32"), ("sigmoid", 15.5, 16.0, "f16"), ("sigmoid", 15.5, 16.0, "bf16"), ("softmax", 0.0, 2.0 ** -30, "f32"),
    ("softmax", 0.0, 2.0 ** -30, "bf16"), ("softmax", 0.0, 2.0 ** -24, "f16"), ("sigmoid", 0.3, 0.3 + 2.0 ** -25, "f32"),
    ("softmax", 0.3, 0.3 + 2.0 ** -25, "f32")])
@pytest.mark.parametrize("experts", [3, 8, 16, 64, 256, 257, 1000])
def test_route_tie_at_the_border_before_a_larger_score(experts, score, low, high, dtype):
    """The last expert that is chosen and the first that is left out have equal logits, and a later one's score is larger by less than
    fp32 shows.  Several ties and several places; every other row of the warp is far from any tie."""
    far = -8.0 if score == "sigmoid" else -20.0
    for top_k in (1, 2):
        rows = []
        g = gen(experts + top_k)
        for r in range(24):
            row = torch.linspace(far - 4, far, experts).double()
            if r % 4 != 3:
                place = torch.randperm(experts, generator=g)[:min(experts, top_k + 2 + r % 3)].sort().values
                row[place] = low
                row[place[-1]] = high
            rows.append(row)
        logits = torch.stack(rows).to(DT[dtype])
        assert (logits.double() == torch.tensor(high, dtype=torch.float32).to(DT[dtype]).double()).any()
        check_choice(logits, top_k, score, torch.zeros(experts))


@pytest.mark.parametrize("experts", [8, 64, 256, 1024])
@pytest.mark.parametrize("top_k", [1, 2, 8])
@pytest.mark.parametrize("around,spread", [(12.0, 2.0), (0.0, 5.0), (8.0, 3.0), (0.0, 0.0)])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_route_of_saturated_scores(experts, top_k, around, spread, groups, kept):
    """bf16 logits, many of them equal, whose sigmoids are nearly 1; and all equal."""
    top_k = min(top_k, experts // groups * kept)
    logits = (around + spread * normal(gen(experts), 300, experts)).clamp(-25, 25).to(torch.bfloat16)
    check_choice(logits, top_k, "sigmoid", torch.zeros(experts), groups, kept)


def test_route_tie_at_the_border_of_biased_scores():
    """Equal logits with equal biases at the border; behind them another bias makes up for a lower logit."""
    logits = torch.full((40, 64), -6.0)
    bias = torch.full((64,), 0.25)
    logits[:, 5] = logits[:, 9] = 0.5
    logits[:, 33] = 0.25
    # the sum is larger than that of 5 and 9 by 2^-26 and some rounding, in fp32 the same
    s = lambda v: 1 / (1 + math.exp(-v))  # noqa: E731
    bias[5] = bias[9] = 0.0
    bias[33] = torch.tensor(s(0.5) - s(0.25), dtype=torch.float64).float()
    for more in range(8):
        check_choice(logits, 1, "sigmoid", bias)
        bias[33] = torch.nextafter(bias[33], torch.tensor(1.0))


# ------------------------------------------------------------------ gradients of very different size in fp16
@pytest.mark.parametrize("hq,hk,d,sizes_q,sizes_k", [(2, 2, 64, [900, 900], None), (4, 2, 128, [300, 500], None), (2, 1, 32, [3000, 200], None),
                                                     (4, 2, 64, [3, 2], [4000, 900]), (2, 2, 40, [4000, 70], [150, 30]), (2, 2, 36, [200, 200], None)])
def test_attention_gradients_of_segments_and_heads_apart_in_fp16(hq, hk, d, sizes_q, sizes_k):
    """dout and v of one segment, of rows of no segment and of another head are larger by up to 2^25 each: every segment and key
    head keeps the digits that it has alone."""
    g = gen(d + sum(sizes_q))
    outside = 5
    seg = [outside + sum(sizes_q[:i]) for i in range(len(sizes_q) + 1)]
    seg_k = seg if sizes_k is None else [outside + sum(sizes_k[:i]) for i in range(len(sizes_k) + 1)]
    nq, nk = seg[-1] + outside, seg_k[-1] + outside
    q, k, v, dout = (normal(g, n, h, d) for n, h in ((nq, hq), (nk, hk), (nk, hk), (nq, hq)))
    per = hq // hk
    dout[:seg[1]] *= 2.0 ** 12
    dout[seg[1]:] *= 2.0 ** -10
    dout[:, per:] *= 2.0 ** -4  # the second key head's queries
    dout[:outside] = dout[-outside:] = 6e4
    v[:outside] = v[-outside:] = -6e4
    q, k, v, dout = (t.half() for t in (q, k, v, dout))
    t_seg, t_seg_k = offsets(*seg), None if seg_k is seg else offsets(*seg_k)
    o, lse = spc.spc_attention_fwd(to(q), to(k), to(v), t_seg, seg_k=t_seg_k)
    args = to(dout), to(q), to(k), to(v), o, lse, t_seg
    grads = spc.spc_attention_bwd(*args, seg_k=t_seg_k)
    again = spc.spc_attention_bwd(*args, seg_k=t_seg_k)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    for s in range(len(sizes_q)):
        a, b = slice(seg[s], seg[s + 1]), slice(seg_k[s], seg_k[s + 1])
        for h in range(hk):
            hs = slice(h * per, h * per + per), slice(h, h + 1)
            own = [0, a.stop - a.start], [0, b.stop - b.start]
            want, bound = ref.attention_bwd(dout[a, hs[0]], q[a, hs[0]], k[b, hs[1]], v[b, hs[1]], o[a, hs[0]].cpu(), lse[a, hs[0]].cpu(), *own,
                                            d ** -0.5, d % 8 == 0)
            for got, w, e, rows, heads, name in zip(grads, want, bound, (a, b, b), (hs[0], hs[1], hs[1]), ("dq", "dk", "dv")):
                # the reference's own allowance of 2^-30 is for values of order 1
                close(got[rows, heads], w, e - 2.0 ** -30, f"{name} of segment {s}, key head {h}")
    for got, n in zip(grads, (nq, nk, nk)):
        assert not got[:outside].any() and not got[n - outside:].any()


# ------------------------------------------------------------------ rows whose values are nearly the same
def norm_of_near_values(x, ga, be, eps):
    """y, mean, rstd and their bounds where a row's mean is far from its spread.

    The first mean is off by f = h mean|x| at most, h = (c / 512 + 64) E as in block_ref.  Differences from it round by E of themselves,
    and their own mean, which is taken off again, by h of their mean size.  The sum of their squares is off by h and a few
    roundings of itself, and so is what is taken off it.  A row whose mean is within 16 spreads of
    zero (256 in 16 bits; give or take a tenth) keeps f."""
    c = x.shape[1]
    (y, mean, rstd), _ = ref.layer_norm_fwd(x, ga, be, eps)
    spreads = 16 if x.dtype is torch.float32 else 256
    x, ga = x.double(), ga.double()
    far = (x - mean[:, None]).abs()
    h = (c / 512 + 64) * E
    f = h * x.abs().mean(1)
    size = far.mean(1) + f
    var = (far ** 2).mean(1)
    kept = torch.where(mean ** 2 < 1.2 * spreads ** 2 * var, f, 0.0)
    off = 2 * E * (far + f[:, None]) + ((h + 2 * E) * size + kept)[:, None]
    vb = 2 * (h + 6 * E) * (var + f * f) + 2 * f * (h + 2 * E) * size + kept ** 2
    rb = vb / (var + eps) + 4 * E
    xh = far * rstd[:, None]
    yb = (off * rstd[:, None] * 1.01 + xh * rb[:, None]) * ga.abs() + 3 * E * xh * ga.abs() + E * y.abs()
    return (y, mean, rstd), (yb + 1e-30, 2 * E * mean.abs() + (h + 2 * E) * size + kept, rstd * rb)


CHANNELS = [5, 24, 64, 333, 334, 512, 1000, 1027, 4001, 8192, 16384, 20000]


@pytest.mark.parametrize("c", CHANNELS)
@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_of_equal_values(c, dtype):
    """Rows of one value: y is beta."""
    x = torch.tensor([30000.0, -1000.3, 0.1, 7.7, 0.0, 123.456, 65000.0])[:, None].expand(7, c).to(DT[dtype])
    ga, be = 1 + 0.3 * normal(gen(c), c), 0.3 * normal(gen(c + 1), c)
    want, bound = norm_of_near_values(x, ga, be, 1e-5)
    got = spc.spc_layer_norm_fwd(to(x), to(ga), to(be))
    close(got[0], want[0], bound[0] + ref.rounding(want[0], DT[dtype]), "y")
    close(got[1], want[1], bound[1], "mean")
    close(got[2], want[2], bound[2], "rstd")


@pytest.mark.parametrize("c", CHANNELS)
@pytest.mark.parametrize("mean,std", [(1000.3, 0.01), (1e6, 1.0), (-3e4, 0.1), (0.0, 1.0)])
def test_layer_norm_of_a_small_spread_far_from_zero(c, mean, std):
    x = (mean + std * torch.randn(40, c, generator=gen(c), dtype=torch.float64)).float()
    ga, be = 1 + 0.3 * normal(gen(c), c), 0.3 * normal(gen(c + 1), c)
    want, bound = norm_of_near_values(x, ga, be, 1e-5)
    got = spc.spc_layer_norm_fwd(to(x), to(ga), to(be))
    for a, w, b, name in zip(got, want, bound, ("y", "mean", "rstd")):
        close(a, w, b, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_of_values_whose_squares_fp32_does_not_hold(dtype):
    """rstd is 0 then, and y beta."""
    x = torch.tensor([1e25, -1e25, 3e24, 0.0] * 10).repeat(3, 1).to(DT[dtype])
    y, mean, rstd = spc.spc_layer_norm_fwd(to(x), None, None)
    assert not y.any() and not rstd.any() and mean.isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", CHANNELS)
def test_layer_norm_of_a_row_does_not_hang_on_its_neighbours(c, dtype):
    """Bits of rows near zero are the same among rows far from it, in place too."""
    x = normal(gen(c), 41, c, dtype=dtype)
    ga, be = 1 + 0.3 * normal(gen(c), c), 0.3 * normal(gen(c + 1), c)
    want = spc.spc_layer_norm_fwd(to(x), to(ga), to(be))
    mixed = to(x).clone()
    mixed[1::3] += 20000  # in bf16 of one or two values
    far = spc.spc_layer_norm_fwd(mixed[1::3].contiguous(), to(ga), to(be))
    for out in (None, mixed):
        got = spc.spc_layer_norm_fwd(mixed, to(ga), to(be), out=out)
        for a, b, f in zip(got, want, far):
            for first in (0, 2):
                assert torch.equal(a[first::3], b[first::3])
            assert torch.equal(a[1::3], f)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c", [5, 24, 40, 333, 334, 1000, 1027, 4100, 8190])
def test_layer_norm_gradient_where_mean_times_rstd_passes_fp32(c, dtype):
    """Rows of one large value: their differences from the mean are 0, and nothing past a row's end takes part."""
    g = gen(c)
    x, dy = torch.full((9, c), 2.0 ** 112).to(DT[dtype]), normal(g, 9, c, dtype=dtype)
    ga = 1 + 0.3 * normal(g, c)
    mean, rstd = torch.full((9,), 2.0 ** 112), torch.full((9,), 2.0 ** 20)
    x[4:], mean[4:], rstd[4:] = normal(g, 5, c, dtype=dtype), 0.1, 0.9
    want, bound = ref.layer_norm_bwd(dy, x, ga, mean, rstd)
    got = spc.spc_layer_norm_bwd(to(dy), to(x), to(ga), to(mean), to(rstd))
    for a, w, b, name in zip(got, want, bound, ("dx", "dgamma", "dbeta")):
        close(a, w, b, name)


# ------------------------------------------------------------------ calls that are refused
def test_attention_refuses_heads_of_no_channels():
    x = torch.zeros(4, 2, 0, device=dev())
    for scale in (None, 1.0):
        with pytest.raises(spc.SpcError):
            spc.spc_attention_fwd(x, x, x, offsets(0, 4), scale=scale)
        with pytest.raises(spc.SpcError):
            spc.spc_attention_bwd(x, x, x, x, x, torch.zeros(4, 2, device=dev()), offsets(0, 4), scale=scale)


def test_choices_that_32_bits_do_not_hold_are_refused():
    """Not taken for their low halves: 2^32 + 1 groups are not one."""
    x = torch.randn(5, 16, device=dev())
    for bad in (dict(groups=2 ** 32 + 1), dict(groups=2, top_groups=2 ** 32 + 1), dict(score=2 ** 32), dict(groups=1 - 2 ** 32)):
        with pytest.raises(spc.SpcError):
            spc.spc_route_fwd(x, 2, **bad)
    expert, gate = spc.spc_route_fwd(x, 2)
    with pytest.raises(spc.SpcError):
        spc.spc_route_bwd(gate, x, expert, score=2 ** 32)


def test_rows_of_more_channels_than_32_bits_hold_are_refused():
    """Not taken for rows of 8 channels, with the rest left as it was."""
    n = 2 ** 32 + 8
    x = torch.zeros(1, n, dtype=torch.float16, device=dev())
    with pytest.raises(spc.SpcError):
        spc.spc_layer_norm_fwd(x, None, None)
    with pytest.raises(spc.SpcError):
        spc.spc_route_fwd(x, 2)
    coords, steps = torch.zeros(1, 4, dtype=torch.int32, device=dev()), spc.spc_rope_steps((1, 1, 1))
    for heads, d in ((1, n), (n // 8, 8)):
        with pytest.raises(spc.SpcError):
            spc.spc_rope_fwd(x.view(1, heads, d), coords, steps, (1, 1, 1))
    for heads, d in ((1, n), (n, 1)):
        q = x.view(1, heads, d)
        with pytest.raises(spc.SpcError):
            spc.spc_attention_fwd(q, q, q, offsets(0, 1))
