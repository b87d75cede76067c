"""GPU parity of the layers between convolutions against plain float64 forms.

Bounds are per element and come from the arithmetic, not from results.  With u the
unit roundoff of the output type (one rounding) and e = 2^-24 that of fp32:
  group norm   sums of N terms are formed in runs of at most N / 256 + 32 additions,
               so a mean is off by h mean|x - pivot| with h = (N / 256 + 32) e and rstd by
               2 h + 8 e relative; an element follows to first order.  exp and the
               division in the activation add 2^-19 relative.
  products     K fp32 accumulations of exact products: K 2^-23 sum|a b| (the factor two
               covers accumulators that truncate).
  dropout      one multiplication and one addition in fp32.
"""

import numpy as np
import pytest
import torch

import layers_ref as ref
import sparse_convolution_hash_gb300 as spc
from gpu_util import DT, dev

pytestmark = pytest.mark.gpu

ACT = {"none": 0, "relu": 1, "silu": 2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def to_dev(a):
    if a is None:
        return None
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).to(dev())


def make_ids(g, n, segments, kind):
    if kind == "one":
        return np.full(n, segments - 1, np.int32)
    if kind == "sorted":
        return np.sort(g.integers(0, segments, n)).astype(np.int32)
    ids = g.integers(0, segments, n).astype(np.int32)
    if kind == "out":  # some rows of no segment, on either side of the range
        ids[g.random(n) < 0.2] = -1
        ids[g.random(n) < 0.1] = segments + 3
    return ids


def close(got, want, bound, what=""):
    got = got.double().cpu()
    bad = (got - want).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, worst {((got - want).abs() - bound).max():.3g}"


# -------------------------------------------------------------------- segments
@pytest.mark.parametrize("kind", ["random", "sorted", "one", "out"])
@pytest.mark.parametrize("n,segments", [(1, 1), (2, 5), (31, 2), (257, 1024), (1024, 3), (5000, 64),
                                        (40001, 300), (160001, 2), (300000, 255), (70000, 1024),
                                        (16384, 70), (16385, 70), (700001, 5), (640000, 1024)])
def test_row_segments(n, segments, kind):
    g = np.random.default_rng(n + segments)
    ids = make_ids(g, n, segments, kind)
    seg, order = spc.spc_row_segments(to_dev(ids), segments)
    want_seg, want_order = ref.segments(ids, segments)
    assert np.array_equal(seg.cpu().numpy(), want_seg)
    assert np.array_equal(order.cpu().numpy(), want_order)
    only, none = spc.spc_row_segments(to_dev(ids), segments, with_order=False)
    assert none is None and torch.equal(only, seg)


def test_row_segments_reads_a_coordinate_column_and_no_rows():
    g = np.random.default_rng(3)
    coords = g.integers(0, 5, (3001, 4)).astype(np.int32)
    seg, order = spc.spc_row_segments(to_dev(coords)[:, 0], 5)
    want = ref.segments(coords[:, 0], 5)
    assert np.array_equal(seg.cpu().numpy(), want[0]) and np.array_equal(order.cpu().numpy(), want[1])
    seg, order = spc.spc_row_segments(to_dev(np.zeros(0, np.int32)), 3)
    assert seg.tolist() == [0, 0, 0, 0] and order.numel() == 0


# ------------------------------------------------------------------ group norm
def norm_case(n, c, groups, segments, kind, dtype, shuffled, seed=0, shift=1.0, affine=True):
    g = np.random.default_rng(seed + n + c)
    ids = make_ids(g, n, segments, kind)
    if not shuffled:
        ids = np.sort(np.where((ids < 0) | (ids >= segments), segments, ids)).astype(np.int32)
    seg, order = ref.segments(ids, segments)
    x = torch.from_numpy(g.standard_normal((n, c)) * g.uniform(0.5, 2, c) + shift * g.standard_normal(c)).to(DT[dtype])
    gamma = torch.from_numpy(1 + 0.3 * g.standard_normal(c)).float() if affine else None
    beta = torch.from_numpy(0.3 * g.standard_normal(c)).float() if affine else None
    dy = torch.from_numpy(g.standard_normal((n, c))).to(DT[dtype])
    return x, dy, gamma, beta, seg, order if shuffled else None


def norm_bound(x, gamma, seg, order, groups, mean, rstd, z, y, dtype):
    """Element bounds of y, and of mean and rstd."""
    n, c = x.shape
    per = c // groups
    counts = np.diff(seg).astype(np.int64) * per
    h = torch.from_numpy((counts / 256 + 32) * ref.EPS32)[:, None]
    spread = torch.zeros_like(mean)
    xh_b = torch.zeros(n, c, dtype=torch.float64)
    for s in range(len(seg) - 1):
        at = ref.positions(seg, order, s)
        if len(at) == 0:
            continue
        v = x[at].double().view(len(at), groups, per)
        # distances from a pivot that is one of the values
        spread[s] = 2 * (v - mean[s][:, None]).abs().amax((0, 2)) + ref.EPS32 * mean[s].abs()
        xh = ((v - mean[s][:, None]) * rstd[s][:, None]).abs()
        e = (h[s] * spread[s] * rstd[s])[:, None] + xh * (2 * h[s] + 2.0 ** -20)[:, None] * (1 + (spread[s] * rstd[s]) ** 2)[:, None]
        e = e + ref.EPS32 * 4 * (v.abs() * rstd[s][:, None] + (mean[s] * rstd[s]).abs()[:, None])
        xh_b[at] = e.reshape(len(at), c)
    ga = torch.ones(c, dtype=torch.float64) if gamma is None else gamma.double().abs()
    y_b = ref.U[DT[dtype]] * y.abs() + 1.2 * (xh_b * ga + 4 * ref.EPS32 * z.abs()) + 2.0 ** -19 * y.abs() + 2.0 ** -24
    return y_b, h * spread + 2 * ref.EPS32 * mean.abs() + 1e-30, rstd * (2 * h * (1 + (spread * rstd) ** 2) + 2.0 ** -20)


NORM = [  # n, c, groups, segments, keys, shuffled
    (1, 1, 1, 1, "random", False), (1, 16, 4, 3, "random", False), (7, 40, 5, 3, "random", True),
    (300, 64, 32, 4, "sorted", False), (1025, 16, 16, 2, "out", True), (999, 33, 11, 5, "out", False),
    (2500, 96, 1, 21, "random", True), (513, 130, 13, 2, "random", False), (4000, 8, 2, 1, "one", False),
    (700, 512, 32, 3, "random", False), (260, 1030, 2, 2, "random", True), (64, 24, 3, 100, "random", False),
    (3000, 72, 3, 2, "one", True), (90, 2048, 64, 2, "random", False), (50, 6000, 4, 2, "random", False)]


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,groups,segments,kind,shuffled", NORM)
def test_group_norm_forward(n, c, groups, segments, kind, shuffled, dtype, act):
    x, _, gamma, beta, seg, order = norm_case(n, c, groups, segments, kind, dtype, shuffled)
    want, mean_r, rstd_r, z = ref.norm_fwd(x, gamma, beta, seg, order, groups, 1e-5, act)
    st = spc.new_status(dev())
    y, mean, rstd = spc.spc_group_norm_fwd(to_dev(x), to_dev(gamma), to_dev(beta), to_dev(seg), groups,
                                           order=to_dev(order), act=ACT[act], status=st)
    spc.check_status(st)
    yb, mb, rb = norm_bound(x, gamma, seg, order, groups, mean_r, rstd_r, z, want, dtype)
    close(mean, mean_r, mb, "mean")
    close(rstd, rstd_r, rb, "rstd")
    close(y, want, yb, "y")
    again = spc.spc_group_norm_fwd(to_dev(x), to_dev(gamma), to_dev(beta), to_dev(seg), groups,
                                   order=to_dev(order), act=ACT[act])
    assert all(torch.equal(p, q) for p, q in zip(again, (y, mean, rstd)))
    # in place
    xd = to_dev(x).clone()
    assert torch.equal(spc.spc_group_norm_fwd(xd, to_dev(gamma), to_dev(beta), to_dev(seg), groups,
                                              order=to_dev(order), act=ACT[act], out=xd)[0], y)


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,groups,segments,kind,shuffled", NORM)
def test_group_norm_backward(n, c, groups, segments, kind, shuffled, dtype, act):
    x, dy, gamma, beta, seg, order = norm_case(n, c, groups, segments, kind, dtype, shuffled)
    _, mean, rstd, z = ref.norm_fwd(x, gamma, beta, seg, order, groups, 1e-5, act)
    mean, rstd = mean.float(), rstd.float()
    dx_r, dg_r, db_r = ref.norm_bwd(dy, x, gamma, beta, mean, rstd, seg, order, groups, act)
    st = spc.new_status(dev())
    args = (to_dev(dy), to_dev(x), to_dev(gamma), to_dev(beta), to_dev(mean), to_dev(rstd), to_dev(seg), groups)
    dx, dg, db = spc.spc_group_norm_bwd(*args, order=to_dev(order), act=ACT[act], status=st)
    spc.check_status(st)
    # an element's terms: xh is off by a few roundings of x, mean and their product with
    # rstd, dz by that times the slope's own slope (below 1.1 for silu) and 2^-18
    per, S = c // groups, len(seg) - 1
    of = torch.full((n,), S, dtype=torch.int64)
    for s in range(S):
        of[ref.positions(seg, order, s)] = s
    pad = lambda t: torch.cat([t.double(), torch.zeros(1, groups, dtype=torch.float64)]).repeat_interleave(per, 1)[of]
    xh = (x.double() - pad(mean)) * pad(rstd)
    d_xh = 4 * ref.EPS32 * ((x.double().abs() + pad(mean).abs()) * pad(rstd))
    sl = ref.slope(z, act).abs()
    d_dz = dy.double().abs() * (sl * 2.0 ** -18 + (1.1 * (d_xh * gamma.double().abs() + 4 * ref.EPS32 * z.abs()) if act == "silu" else 0) + 2.0 ** -22)
    if act == "relu":  # an element at the kink may fall on either side
        d_dz = torch.where(z.abs() < 1e-4, dy.double().abs(), d_dz)
    ga = gamma.double().abs()
    dz = dy.double().abs() * sl
    counts = torch.from_numpy(np.concatenate([np.diff(seg), [0]]).astype(np.float64) * per).clamp(min=1)
    h = ((counts / 256 + 32) * ref.EPS32)[of][:, None]
    inside = (of < S).double()[:, None]

    def seg_mean(v):  # mean of |v| over the element's (segment, group), spread back
        t = torch.zeros(S + 1, c, dtype=torch.float64).index_add_(0, of, v)
        t = t.view(S + 1, groups, per).sum(2) / counts[:, None]
        return t.repeat_interleave(per, 1)[of]

    a_abs, b_abs = seg_mean(dz * ga), seg_mean(dz * ga * xh.abs())
    d_a = seg_mean(d_dz * ga) + h * a_abs
    d_b = seg_mean(d_dz * ga * xh.abs() + dz * ga * d_xh) + h * b_abs
    d_dx = pad(rstd) * (ga * d_dz + d_a + xh.abs() * d_b + d_xh * b_abs + 8 * ref.EPS32 * (ga * dz + a_abs + xh.abs() * b_abs))
    close(dx, dx_r, ref.U[DT[dtype]] * dx_r.abs() + d_dx * 1.05 * inside + 2.0 ** -24, "dx")
    hn = (n / 256 + 32 + S) * ref.EPS32
    close(dg, dg_r, ((d_dz * xh.abs() + dz * d_xh + hn * dz * xh.abs()) * inside).sum(0) * 1.05 + 1e-30, "dgamma")
    close(db, db_r, ((d_dz + hn * dz) * inside).sum(0) * 1.05 + 1e-30, "dbeta")
    again = spc.spc_group_norm_bwd(*args, order=to_dev(order), act=ACT[act])
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dg, db)))


def test_group_norm_gradient_is_the_difference_of_the_forward():
    x, dy, gamma, beta, seg, order = norm_case(400, 24, 3, 3, "random", "f32", True)
    _, mean, rstd, _ = ref.norm_fwd(x, gamma, beta, seg, order, 3, 1e-5, "silu")
    grads = spc.spc_group_norm_bwd(to_dev(dy), to_dev(x), to_dev(gamma), to_dev(beta), to_dev(mean.float()),
                                   to_dev(rstd.float()), to_dev(seg), 3, order=to_dev(order), act=2)
    args = [x.double(), gamma.double(), beta.double()]
    torch.manual_seed(0)
    for k, grad in enumerate(grads):
        v = torch.randn_like(args[k])
        h = 1e-5
        vals = []
        for sign in (1, -1):
            moved = list(args)
            moved[k] = args[k] + sign * h * v
            vals.append(float((dy.double() * ref.norm_fwd(*moved, seg, order, 3, 1e-5, "silu")[0]).sum()))
        want = (vals[0] - vals[1]) / (2 * h)
        got = (grad.double().cpu() * v).sum()
        # 1e-6 relative in each of the summed terms (fp32 gradients)
        assert abs(want - float(got)) < 1e-5 * float((grad.double().cpu() * v).abs().sum())


@pytest.mark.parametrize("n,first", [(2000, 0.0), (2000, 1e4), (40000, 0.0)])
def test_group_norm_far_from_zero(n, first):
    """Features at 1000 +- 1 with a first row elsewhere: the variance keeps its digits."""
    g = np.random.default_rng(0)
    x = torch.from_numpy(1000 + g.standard_normal((n, 16))).float()
    x[0] = first
    seg = np.array([0, n], np.int32)
    y_r, mean_r, rstd_r, _ = ref.norm_fwd(x, None, None, seg, None, 4, 1e-5, "none")
    y, mean, rstd = spc.spc_group_norm_fwd(to_dev(x), None, None, to_dev(seg), 4)
    # the values' own distances from the mean are exact to 1000 e / spread; 1e-4 covers
    # that and the sums of 256-element runs around a pivot, where a one-pass sum of
    # squares would be off by (1000 / spread)^2 e N^(1/2) or more
    assert float((rstd.double().cpu() / rstd_r - 1).abs().max()) < 1e-4
    assert float((mean.double().cpu() / mean_r - 1).abs().max()) < 1e-6
    assert float((y.double().cpu() - y_r).norm() / y_r.norm()) < 1e-3


def test_group_norm_constant_rows_nan_and_inf():
    n, c = 600, 32
    g = np.random.default_rng(1)
    seg = np.array([0, 200, 400, 600], np.int32)
    x = torch.from_numpy(g.standard_normal((n, c))).float()
    x[:200] = 3.25          # variance 0
    x[450, 3] = float("nan")  # only its own segment and group suffer
    x[500, 9] = float("inf")
    y, mean, rstd = spc.spc_group_norm_fwd(to_dev(x), None, None, to_dev(seg), 8, act=1)
    y, rstd = y.cpu(), rstd.cpu()
    assert y[:200].abs().max() == 0 and torch.allclose(rstd[0], torch.full((8,), 1e-5) ** -0.5)
    assert torch.isfinite(y[200:400]).all()
    bad = torch.isnan(y[400:]).all(0).view(8, 4).all(1)
    assert bad.tolist() == [True, False, True, False, False, False, False, False]
    assert torch.isfinite(y[400:].view(200, 8, 4)[:, ~bad]).all()


def test_group_norm_no_rows_and_empty_segments():
    seg = to_dev(np.zeros(4, np.int32))
    for dt in (torch.float32, torch.bfloat16):
        x = torch.empty(0, 16, device=dev(), dtype=dt)
        y, mean, rstd = spc.spc_group_norm_fwd(x, None, None, seg, 4)
        assert y.shape == (0, 16) and mean.abs().max() == 0
        assert torch.allclose(rstd, torch.full_like(rstd, 1e-5) ** -0.5)
        dx, dg, db = spc.spc_group_norm_bwd(x, x, None, None, mean, rstd, seg, 4)
        assert dx.shape == (0, 16) and dg.abs().max() == 0 and db.abs().max() == 0


def test_group_norm_reports_bad_offsets_and_rows():
    x = torch.randn(100, 16, device=dev())
    for seg in ([0, 60, 40, 100], [0, 50, 100, 120], [-5, 10, 20, 30]):
        st = spc.new_status(dev())
        spc.spc_group_norm_fwd(x, None, None, to_dev(np.array(seg, np.int32)), 4, status=st)
        with pytest.raises(spc.SpcError) as e:
            spc.check_status(st)
        assert e.value.code == 10
    seg = to_dev(np.array([0, 100], np.int32))
    for bad in (-1, 100, 2 ** 31 - 1):
        order = np.arange(100, dtype=np.int32)
        order[17] = bad
        st = spc.new_status(dev())
        spc.spc_group_norm_fwd(x, None, None, seg, 4, order=to_dev(order), status=st)
        assert int(st) == 10
        st.zero_()
        m = torch.zeros(1, 4, device=dev())
        spc.spc_group_norm_bwd(x, x, None, None, m, m + 1, seg, 4, order=to_dev(order), status=st)
        assert int(st) == 10


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_norm_unaligned_views(dtype):
    """Tensors that start off a 16-byte boundary give the same values."""
    x, dy, gamma, beta, seg, _ = norm_case(500, 32, 8, 2, "sorted", dtype, False)
    want = spc.spc_group_norm_fwd(to_dev(x), to_dev(gamma), to_dev(beta), to_dev(seg), 8, act=2)
    room = torch.empty(500 * 32 + 1, device=dev(), dtype=DT[dtype])[1:].view(500, 32)
    room.copy_(to_dev(x))
    got = spc.spc_group_norm_fwd(room, to_dev(gamma), to_dev(beta), to_dev(seg), 8, act=2)
    tol = 4 * ref.U[DT[dtype]]
    for p, q in zip(got, want):
        assert torch.allclose(p.double(), q.double(), rtol=tol, atol=tol)
    room2 = torch.empty(500 * 32 + 1, device=dev(), dtype=DT[dtype])[1:].view(500, 32)
    room2.copy_(to_dev(dy))
    a = spc.spc_group_norm_bwd(room2, room, to_dev(gamma), to_dev(beta), *want[1:], to_dev(seg), 8, act=2)
    b = spc.spc_group_norm_bwd(to_dev(dy), to_dev(x), to_dev(gamma), to_dev(beta), *want[1:], to_dev(seg), 8, act=2)
    for p, q in zip(a, b):
        assert torch.allclose(p.double(), q.double(), rtol=tol, atol=max(tol, 1e-4))


# --------------------------------------------------------------------- dropout
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,skip", [(1, 0), (3, 0), (8, 0), (1037, 0), (4099, 1)])
def test_dropout(n, skip, dtype, p, residual):
    g = np.random.default_rng(n)
    room = torch.from_numpy(g.standard_normal(n + skip)).to(DT[dtype])
    x = to_dev(room)[skip:]
    res = to_dev(torch.from_numpy(g.standard_normal(n + skip)).to(DT[dtype]))[skip:] if residual else None
    seed, offset = 0x1234567890ABCDEF, 0x0FEDCBA987654321
    rng = to_dev(torch.tensor([seed, offset]))
    y = spc.spc_dropout_fwd(x, p, rng, residual=res)
    keep = torch.from_numpy(ref.dropout_words(seed, offset, 0, n) >= np.uint64(round(p * 2 ** 32)))
    xd = x.double().cpu()
    base = res.double().cpu() if residual else torch.zeros(n, dtype=torch.float64)
    want = base + torch.where(keep, xd / (1 - p) if p < 1 else xd * 0, torch.zeros_like(xd))
    mag = base.abs() + torch.where(keep, xd.abs() / (1 - p) if p < 1 else xd * 0, torch.zeros_like(xd))
    close(y, want, ref.U[DT[dtype]] * want.abs() + 3 * ref.EPS32 * mag + 2.0 ** -25)
    if not residual:
        assert torch.equal(y.cpu() == 0, ~keep | (xd == 0))
        assert torch.equal(spc.spc_dropout_bwd(x, p, rng), y)
    xc = x.clone()
    assert torch.equal(spc.spc_dropout_fwd(xc, p, rng, residual=res, out=xc), y)


def test_dropout_drops_nan_and_inf_and_moves_with_its_offset():
    n = 4096
    x = torch.full((n,), float("nan"), device=dev())
    x[::2] = float("inf")
    rng = to_dev(torch.tensor([5, 6]))
    y = spc.spc_dropout_fwd(x, 0.5, rng)
    keep = torch.from_numpy(ref.dropout_words(5, 6, 0, n) >= np.uint64(2 ** 31))
    assert (y.cpu()[~keep] == 0).all() and not torch.isfinite(y.cpu()[keep]).any()
    one = torch.ones(n, device=dev())
    a, b = spc.spc_dropout_fwd(one, 0.5, rng), spc.spc_dropout_fwd(one, 0.5, rng + 1)
    assert 0.4 < float((a != b).float().mean()) < 0.6
    # the kept share of 4096 draws: 0.5 +- 5 sigma
    assert abs(float((a != 0).float().mean()) - 0.5) < 5 * 0.5 / 64


def test_dropout_past_32_bits():
    """More than 2^32 elements: the last ones follow the words of their own indices."""
    n = 2 ** 32 + 4099
    x = torch.ones(n, device=dev(), dtype=torch.bfloat16)
    rng = to_dev(torch.tensor([77, 78]))
    spc.spc_dropout_fwd(x, 0.25, rng, out=x)
    for first in (0, 2 ** 31 - 5, 2 ** 32 - 9, n - 1001):
        keep = torch.from_numpy(ref.dropout_words(77, 78, first, 1000) >= np.uint64(2 ** 30))
        assert torch.equal(x[first:first + 1000].cpu() != 0, keep)


# ------------------------------------------------------------- grouped products
def grouped_case(m, cin, cout, segments, kind, dtype, slots, seed=0):
    g = np.random.default_rng(seed + m + cin + cout)
    ids = make_ids(g, m, segments, kind)
    seg, order = ref.segments(ids, segments)
    n_x = m // slots if slots else m
    x = torch.from_numpy(g.standard_normal((n_x, cin))).to(DT[dtype])
    dy = torch.from_numpy(g.standard_normal((m, cout))).to(DT[dtype])
    w = torch.from_numpy(g.standard_normal((segments, cin, cout)) / np.sqrt(cin)).to(DT[dtype])
    x_rows = (order // slots).astype(np.int32) if slots else None
    return x, dy, w, seg, x_rows, order if slots else None


GROUPED = [  # m, cin, cout, segments, keys, slots (0: rows in grouped order)
    (1, 8, 8, 1, "random", 0), (1, 64, 64, 5, "random", 1), (2, 1, 1, 3, "random", 0), (130, 64, 64, 3, "random", 0),
    (257, 128, 64, 4, "out", 1), (512, 64, 136, 2, "one", 2), (600, 200, 128, 7, "random", 2),
    (777, 100, 72, 5, "out", 0), (1000, 33, 65, 9, "random", 2), (64, 256, 512, 64, "random", 2),
    (1500, 256, 264, 3, "random", 1), (900, 72, 1000, 40, "out", 2), (300, 520, 40, 2, "random", 0),
    (16, 1024, 256, 100, "random", 2), (129, 8, 24, 200, "random", 0), (2600, 128, 384, 2, "one", 1),
    (9000, 264, 264, 3, "random", 0), (9000, 136, 264, 2, "one", 2), (12000, 64, 520, 4, "sorted", 0)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,cin,cout,segments,kind,slots", GROUPED)
def test_grouped_products(m, cin, cout, segments, kind, slots, dtype):
    x, dy, w, seg, x_rows, y_rows = grouped_case(m, cin, cout, segments, kind, dtype, slots)
    st = spc.new_status(dev())
    lists = dict(x_rows=to_dev(x_rows), y_rows=to_dev(y_rows), status=st)
    u = ref.U[DT[dtype]]

    y = spc.spc_grouped_fwd(to_dev(x), to_dev(w), to_dev(seg), **lists)
    want, mag = ref.grouped_fwd(x, w, seg, x_rows, y_rows, m)
    close(y, want, 1.01 * u * want.abs() + cin * 2.0 ** -23 * mag * 1.01 + 2.0 ** -25 * (mag > 0), "y")

    # a token's slots each have a row of dx
    dx = spc.spc_grouped_dgrad(to_dev(dy), to_dev(w), to_dev(seg), x_rows=to_dev(y_rows), y_rows=to_dev(y_rows), status=st)
    want, mag = ref.grouped_fwd(dy, w.transpose(1, 2), seg, y_rows, y_rows, m)
    close(dx, want, 1.01 * u * want.abs() + cout * 2.0 ** -23 * mag * 1.01 + 2.0 ** -25 * (mag > 0), "dx")

    dw = spc.spc_grouped_wgrad(to_dev(x), to_dev(dy), to_dev(seg), **lists)
    want, mag = ref.grouped_wgrad(x, dy, seg, x_rows, y_rows)
    rows = torch.from_numpy(np.diff(seg).astype(np.float64))[:, None, None]
    close(dw, want, rows * 2.0 ** -23 * mag, "dw")
    spc.check_status(st)
    assert torch.equal(y, spc.spc_grouped_fwd(to_dev(x), to_dev(w), to_dev(seg), **lists))
    assert torch.equal(dw, spc.spc_grouped_wgrad(to_dev(x), to_dev(dy), to_dev(seg), **lists))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_gradients_are_differences_of_the_forward(dtype):
    """The forward is linear in x and in W: the difference of two forwards along v is
    exact in float64, so <dx, v> and <dW, v> have to match it to the gradients' rounding."""
    x, dy, w, seg, x_rows, y_rows = grouped_case(300, 64, 72, 4, "random", dtype, 1)
    dx = spc.spc_grouped_dgrad(to_dev(dy), to_dev(w), to_dev(seg), x_rows=to_dev(x_rows), y_rows=to_dev(y_rows))
    dw = spc.spc_grouped_wgrad(to_dev(x), to_dev(dy), to_dev(seg), x_rows=to_dev(x_rows), y_rows=to_dev(y_rows))
    torch.manual_seed(0)
    f = lambda a, b: (dy.double() * ref.grouped_fwd(a, b, seg, x_rows, y_rows, 300)[0]).sum()
    for grad, k in ((dx, 0), (dw, 1)):
        args = [x.double(), w.double()]
        v = torch.randn_like(args[k])
        plus, minus = list(args), list(args)
        plus[k], minus[k] = args[k] + v, args[k] - v
        want = (f(*plus) - f(*minus)) / 2
        terms = (grad.double().cpu() * v)
        assert abs(float(want - terms.sum())) < (ref.U[DT[dtype]] + 72 * 2.0 ** -20) * float(terms.abs().sum())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout", [(64, 128), (100, 33)])
def test_grouped_nan_stays_in_its_rows(cin, cout, dtype):
    """A NaN or infinity in one row (or in an expert's weight) reaches that row (that
    expert) only: what a partial tile reads past its segment has no part in the result."""
    x, dy, w, seg, _, _ = grouped_case(333, cin, cout, 4, "sorted", dtype, 0)
    x[int(seg[1])] = float("nan")      # the first row of expert 1, right after expert 0's tail
    dy[int(seg[2])] = float("inf")
    w[3] = float("nan")
    y = spc.spc_grouped_fwd(to_dev(x), to_dev(w), to_dev(seg)).cpu()
    nan = torch.isnan(y).any(1)
    want = torch.zeros(333, dtype=torch.bool)
    want[int(seg[1])] = True
    want[int(seg[3]):int(seg[4])] = True
    assert torch.equal(nan, want)
    dw = spc.spc_grouped_wgrad(to_dev(x), to_dev(dy), to_dev(seg)).cpu()
    assert torch.isfinite(dw[0]).all() and torch.isfinite(dw[3]).all()
    assert torch.isnan(dw[1]).all() and not torch.isfinite(dw[2]).any()


def test_grouped_no_rows_and_reports():
    d = dev()
    w = torch.randn(3, 64, 64, device=d, dtype=torch.bfloat16)
    none = torch.empty(0, 64, device=d, dtype=torch.bfloat16)
    seg0 = torch.zeros(4, dtype=torch.int32, device=d)
    assert spc.spc_grouped_fwd(none, w, seg0).shape == (0, 64)
    assert spc.spc_grouped_dgrad(none, w, seg0).shape == (0, 64)
    assert spc.spc_grouped_wgrad(none, none, seg0).abs().max() == 0
    x = torch.randn(200, 64, device=d, dtype=torch.bfloat16)
    # no row has an expert
    assert spc.spc_grouped_fwd(x, w, seg0).abs().max() == 0
    assert spc.spc_grouped_wgrad(x, x, seg0).abs().max() == 0
    for dt in (torch.bfloat16, torch.float32):
        xs, ws = x.to(dt), w.to(dt)
        for seg in ([0, 150, 100, 200], [0, 50, 100, 201], [-1, 50, 100, 200]):
            seg = torch.tensor(seg, dtype=torch.int32, device=d)
            for f in (lambda st: spc.spc_grouped_fwd(xs, ws, seg, status=st),
                      lambda st: spc.spc_grouped_dgrad(xs, ws, seg, status=st),
                      lambda st: spc.spc_grouped_wgrad(xs, xs, seg, status=st)):
                st = spc.new_status(d)
                f(st)
                assert int(st) == 10
        seg = torch.tensor([0, 50, 100, 200], dtype=torch.int32, device=d)
        good = torch.arange(200, dtype=torch.int32, device=d)
        for bad in (-1, 200, 2 ** 31 - 1):
            rows = good.clone()
            rows[120] = bad
            ok = spc.spc_grouped_fwd(xs, ws, seg)
            st = spc.new_status(d)
            got = spc.spc_grouped_fwd(xs, ws, seg, x_rows=rows, status=st)
            assert int(st) == 10 and got[120].abs().max() == 0
            keep = good != 120
            assert torch.equal(got[keep], ok[keep])
            for f in (lambda st: spc.spc_grouped_fwd(xs, ws, seg, y_rows=rows, status=st),
                      lambda st: spc.spc_grouped_dgrad(xs, ws, seg, y_rows=rows, status=st),
                      lambda st: spc.spc_grouped_wgrad(xs, xs, seg, x_rows=rows, status=st),
                      lambda st: spc.spc_grouped_wgrad(xs, xs, seg, y_rows=rows, status=st)):
                st = spc.new_status(d)
                f(st)
                assert int(st) == 10


# ------------------------------------------------- streams, graphs, no allocation
def test_layers_on_a_side_stream_and_in_a_graph():
    """Every layer captured once on a side stream with the caller's buffers; replays
    follow the inputs, a dropout mask follows the offset its caller advances."""
    d = dev()
    torch.manual_seed(0)
    n, c = 3000, 64
    ids = torch.randint(0, 4, (n,), device=d, dtype=torch.int32)
    x = torch.randn(n, c, device=d, dtype=torch.bfloat16)
    w = torch.randn(4, c, 128, device=d, dtype=torch.bfloat16) / 8
    gamma, beta = torch.ones(c, device=d), torch.zeros(c, device=d)
    rng = torch.tensor([1, 2], device=d)

    def layers():
        seg, order = spc.spc_row_segments(ids, 4)
        y, mean, rstd = spc.spc_group_norm_fwd(x, gamma, beta, seg, 8, order=order, act=2)
        z = spc.spc_grouped_fwd(y, w, seg, x_rows=order, y_rows=order)
        dz = spc.spc_dropout_fwd(z, 0.3, rng)
        dy = spc.spc_grouped_dgrad(dz, w, seg, x_rows=order, y_rows=order)
        dw = spc.spc_grouped_wgrad(y, dz, seg, x_rows=order, y_rows=order)
        dx, dg, db = spc.spc_group_norm_bwd(dy, x, gamma, beta, mean, rstd, seg, 8, order=order, act=2)
        return [seg, order, y, z, dz, dw, dx, dg, db]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in layers()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = layers()
    side.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    x.mul_(2.0)
    ids.copy_(torch.flip(ids, [0]))
    rng[1] += 1
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, [t.clone() for t in layers()]):
        assert torch.equal(p, q)


def test_binding_checks_of_shapes_and_types():
    d = dev()
    x = torch.randn(10, 16, device=d)
    seg = torch.tensor([0, 10], dtype=torch.int32, device=d)
    w = torch.randn(1, 16, 8, device=d)
    rng = torch.tensor([1, 2], device=d)
    bad = [lambda: spc.spc_group_norm_fwd(x.double(), None, None, seg, 4),
           lambda: spc.spc_group_norm_fwd(x, x[0, :8], None, seg, 4),
           lambda: spc.spc_group_norm_fwd(x, None, None, seg, 4, order=seg),
           lambda: spc.spc_group_norm_fwd(x, None, None, seg, 4, out=x[:5]),
           lambda: spc.spc_group_norm_fwd(x, None, None, seg, 4, out=x.half()),
           lambda: spc.spc_group_norm_bwd(x[:5], x, None, None, x, x, seg, 4),
           lambda: spc.spc_dropout_fwd(x, 0.5, rng[:1]),
           lambda: spc.spc_dropout_fwd(x, 0.5, rng.float()),
           lambda: spc.spc_dropout_fwd(x, 0.5, rng, residual=x[:5]),
           lambda: spc.spc_grouped_fwd(x[:, :8], w, seg),
           lambda: spc.spc_grouped_fwd(x, w, torch.zeros(3, dtype=torch.int32, device=d)),
           lambda: spc.spc_grouped_fwd(x, w, seg, x_rows=seg, y_rows=torch.zeros(3, dtype=torch.int32, device=d)),
           lambda: spc.spc_row_segments(torch.zeros(4, 4, dtype=torch.int32, device=d), 2),
           lambda: spc.spc_row_segments(seg, 2, out=seg)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: spc.spc_group_norm_fwd(x, None, None, seg, 3), lambda: spc.spc_dropout_fwd(x, 1.5, rng),
              lambda: spc.spc_group_norm_fwd(x, None, None, seg, 4, act=7),
              lambda: spc.spc_grouped_fwd(x[:5].contiguous(), w, seg, out=torch.empty(5, 8, device=d), x_rows=None,
                                          y_rows=torch.arange(10, dtype=torch.int32, device=d))):
        with pytest.raises((spc.SpcError, ValueError)):
            f()


def test_wait_limit_ends_the_pipelined_layers_with_a_status():
    """With a limit of 0 a wait whose phase is not complete gives up at once: the kernels report
    it, free what they hold and return, and the same calls work again afterwards."""
    d = dev()
    x = torch.randn(6000, 512, device=d, dtype=torch.bfloat16)
    w = torch.randn(2, 512, 512, device=d, dtype=torch.bfloat16)
    seg = torch.tensor([0, 2500, 6000], dtype=torch.int32, device=d)
    rows = torch.randperm(6000, device=d).to(torch.int32)
    calls = [lambda st: spc.spc_grouped_fwd(x, w, seg, status=st),
             lambda st: spc.spc_grouped_fwd(x, w, seg, x_rows=rows, status=st),
             lambda st: spc.spc_grouped_dgrad(x, w, seg, status=st),
             lambda st: spc.spc_grouped_wgrad(x, x, seg, status=st),
             lambda st: spc.spc_grouped_wgrad(x, x, seg, x_rows=rows, y_rows=rows, status=st),
             lambda st: spc.spc_group_norm_fwd(x, None, None, seg, 32, status=st)[0],
             lambda st: spc.spc_group_norm_bwd(x, x, None, None, torch.zeros(2, 32, device=d), torch.ones(2, 32, device=d),
                                               seg, 32, status=st)[0]]
    want = [f(None).clone() for f in calls]
    old = spc.spc_get_wait_limit_ns()
    try:
        spc.spc_set_wait_limit_ns(0)
        for f in calls:
            st = spc.new_status(d)
            f(st)
            torch.cuda.synchronize()
            assert int(st) == 9  # SPC_ERR_TIMEOUT
    finally:
        spc.spc_set_wait_limit_ns(old)
    for f, y in zip(calls, want):
        st = spc.new_status(d)
        assert torch.equal(f(st), y)
        spc.check_status(st)


def test_layers_past_32_bits():
    """More than 2^31 (and 2^32) elements: rows at the end are addressed as rows at the start."""
    d = dev()
    c = 512
    n = 2 ** 32 // c + 4097
    x = torch.zeros(n, c, device=d, dtype=torch.bfloat16)
    tail = torch.randn(3000, c, device=d).to(torch.bfloat16)
    x[-3000:] = tail
    seg = torch.tensor([0, n - 3000, n], dtype=torch.int32, device=d)
    y, mean, rstd = spc.spc_group_norm_fwd(x, None, None, seg, 32, act=2)
    small = torch.tensor([0, 3000], dtype=torch.int32, device=d)
    want, mean_w, rstd_w = spc.spc_group_norm_fwd(tail, None, None, small, 32, act=2)
    assert torch.allclose(mean[1], mean_w[0], atol=1e-6) and torch.allclose(rstd[1], rstd_w[0], rtol=1e-5)
    assert torch.allclose(y[-3000:].float(), want.float(), rtol=2 ** -7, atol=2 ** -7)
    assert float(y[: n - 3000: 65537].abs().max()) == 0
    dx, dg, db = spc.spc_group_norm_bwd(x, x, None, None, mean, rstd, seg, 32, act=2, out=y)
    dx_w, dg_w, db_w = spc.spc_group_norm_bwd(tail, tail, None, None, mean_w, rstd_w, small, 32, act=2)
    assert torch.allclose(dx[-3000:].float(), dx_w.float(), rtol=2 ** -6, atol=2 ** -6)
    # the rows of zeros add nothing: xh = 0 there and dy = 0
    assert torch.allclose(dg, dg_w, rtol=1e-3, atol=1e-2) and torch.allclose(db, db_w, rtol=1e-3, atol=1e-2)
    del y, dx
    w = torch.randn(2, c, 64, device=d).to(torch.bfloat16)
    z = spc.spc_grouped_fwd(x, w, seg)
    assert torch.equal(z[-3000:], spc.spc_grouped_fwd(tail, w[1:].contiguous(), small))
    dw = spc.spc_grouped_wgrad(x, z, seg)
    dw_w = spc.spc_grouped_wgrad(tail, z[-3000:].contiguous(), small)
    assert float(dw[0].abs().max()) == 0
    assert torch.allclose(dw[1], dw_w[0], rtol=1e-4, atol=1e-2)
    back = spc.spc_grouped_dgrad(z, w, seg, out=x)
    assert torch.equal(back[-3000:], spc.spc_grouped_dgrad(z[-3000:].contiguous(), w[1:].contiguous(), small))
