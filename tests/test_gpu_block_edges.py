"""A transformer block's layers where a call is unusual: waits that run out, rows past 32 bits, other streams,
tensors in other layouts and types, status words and workspaces, results against differences.

Bounds are those of test_gpu_block.py where nothing else is said."""

import math

import pytest
import torch

import block_ref as ref
import sparse_convolution_hash_gb300 as spc
from gpu_util import DT, dev
from test_gpu_block import attn_case, check_attention, close, gen, normal, run_attention, to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def offsets(*seg):
    return torch.tensor(seg, dtype=torch.int32, device=dev())


# ------------------------------------------------------------------ waits that run out
def test_wait_limit_ends_attention_with_a_status():
    """With a limit of 0 a wait whose phase is not complete gives up at once: the kernels report it, free what they hold
    and return, and the same calls work again afterwards."""
    g = gen(3)
    calls = []
    for dtype, sizes, d, hk in (("bf16", [3000, 1000], 64, 2), ("f16", [700, 300], 128, 1), ("bf16", [40] * 60, 32, 2)):
        n = sum(sizes)
        q, k, v = (normal(g, n, h, d, dtype=dtype).to(dev()) for h in (2, hk, hk))
        seg = offsets(*[sum(sizes[:i]) for i in range(len(sizes) + 1)])
        o, lse = spc.spc_attention_fwd(q, k, v, seg)
        calls.append(lambda st, a=(q, k, v, seg): spc.spc_attention_fwd(*a, status=st))
        calls.append(lambda st, a=(o, q, k, v, o, lse, seg): spc.spc_attention_bwd(*a, status=st))
    want = [[t.clone() for t in f(None)] for f in calls]
    old = spc.spc_get_wait_limit_ns()
    try:
        spc.spc_set_wait_limit_ns(0)
        for f in calls:
            st = spc.new_status(dev())
            f(st)
            torch.cuda.synchronize()
            assert int(st) == 9  # SPC_ERR_TIMEOUT
    finally:
        spc.spc_set_wait_limit_ns(old)
    for f, y in zip(calls, want):
        st = spc.new_status(dev())
        assert all(torch.equal(a, b) for a, b in zip(f(st), y))
        spc.check_status(st)


# ------------------------------------------------------------------ past 32 bits
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_rows_past_32_bits(dtype):
    """The last segment's keys lie beyond element 2^32: results are those of the keys alone."""
    hk, d, tail = 16, 128, 300
    nk = 2 ** 32 // (hk * d) + 4000
    g = gen(4)
    q, kt, vt = (normal(g, n, 16, d, dtype=dtype).to(dev()) for n in (70, tail, tail))
    dout = normal(g, 70, 16, d, dtype=dtype).to(dev())
    k, v = (torch.zeros(nk, hk, d, dtype=DT[dtype], device=dev()) for _ in range(2))
    k[-tail:], v[-tail:] = kt, vt
    seg, seg_k = offsets(0, 0, 70), offsets(0, nk - tail, nk)
    st = spc.new_status(dev())
    o, lse = spc.spc_attention_fwd(q, k, v, seg, seg_k=seg_k, status=st)
    small = offsets(0, 70), offsets(0, tail)
    want, want_lse = spc.spc_attention_fwd(q, kt, vt, small[0], seg_k=small[1])
    # the number of splits is the longer call's: sums join in another order
    u = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -18
    assert torch.allclose(o.float(), want.float(), rtol=u, atol=u) and torch.allclose(lse, want_lse, rtol=1e-5, atol=1e-5)
    dq, dk, dv = spc.spc_attention_bwd(dout, q, k, v, o, lse, seg, seg_k=seg_k, status=st)
    spc.check_status(st)
    wq, wk, wv = spc.spc_attention_bwd(dout, q, kt, vt, o, lse, small[0], seg_k=small[1])
    for a, b in ((dq, wq), (dk[-tail:], wk), (dv[-tail:], wv)):
        assert torch.allclose(a.float(), b.float(), rtol=8 * u, atol=8 * u)
    assert not dk[:nk - tail:4099].any() and not dv[:nk - tail:4099].any()


def test_rows_past_32_bits():
    d = dev()
    c = 512
    n = 2 ** 32 // c + 4097
    x = torch.zeros(n, c, device=d, dtype=torch.bfloat16)
    tail = torch.randn(3000, c, device=d).to(torch.bfloat16)
    x[-3000:] = tail
    y, mean, rstd = spc.spc_layer_norm_fwd(x, None, None)
    want, mean_w, rstd_w = spc.spc_layer_norm_fwd(tail, None, None)
    assert torch.equal(y[-3000:], want) and torch.equal(mean[-3000:], mean_w) and torch.equal(rstd[-3000:], rstd_w)
    dx, dg, db = spc.spc_layer_norm_bwd(x, x, None, mean, rstd, out=y)
    dx_w, dg_w, db_w = spc.spc_layer_norm_bwd(tail, tail, None, mean_w, rstd_w)
    assert torch.equal(dx[-3000:], dx_w)
    # the rows of zeros add nothing: sums of 3,000 terms of size 1 in another order
    assert torch.allclose(dg, dg_w, rtol=1e-4, atol=1e-2) and torch.allclose(db, db_w, rtol=1e-4, atol=1e-2)
    del dx, y
    heads = x.view(n, 8, 64)
    coords = torch.zeros(n, 4, dtype=torch.int32, device=d)
    coords[-3000:] = torch.randint(0, 100, (3000, 4), device=d, dtype=torch.int32)
    steps = spc.spc_rope_steps((10, 11, 11))
    turned = spc.spc_rope_fwd(heads, coords, steps, (10, 11, 11))
    assert torch.equal(turned[-3000:], spc.spc_rope_fwd(tail.view(3000, 8, 64), coords[-3000:].contiguous(), steps, (10, 11, 11)))
    del turned
    expert, gate = spc.spc_route_fwd(x, 4)
    e, w = spc.spc_route_fwd(tail, 4)
    assert torch.equal(expert[-3000:], e) and torch.equal(gate[-3000:], w) and expert[0].tolist() == [0, 1, 2, 3]
    dl = spc.spc_route_bwd(gate, x, expert)
    assert torch.equal(dl[-3000:], spc.spc_route_bwd(w, tail, e))


# ------------------------------------------------------------------ layouts and types
def test_attention_takes_other_layouts():
    """Copies are made of what the kernels do not read in place: heads apart, broadcast and transposed tensors, other types."""
    g = gen(5)
    n, h, d = 150, 2, 32
    q, k, v = (normal(g, n, h, d, dtype="bf16").to(dev()) for _ in range(3))
    dout = normal(g, 1, h, d, dtype="bf16").to(dev()).expand(n, h, d)
    seg = offsets(0, 80, 150)
    want = spc.spc_attention_fwd(q, k, v, seg)
    grads = spc.spc_attention_bwd(dout.contiguous(), q, k, v, *want, seg)
    apart = torch.zeros(h, n, d, dtype=torch.bfloat16, device=dev())
    apart.copy_(q.transpose(0, 1))
    got = spc.spc_attention_fwd(apart.transpose(0, 1), k.float(), v.half().float(), seg.long())
    ref_v = spc.spc_attention_fwd(q, k, v.half().float().to(torch.bfloat16), seg)
    assert all(torch.equal(a, b) for a, b in zip(got, ref_v))
    got = spc.spc_attention_bwd(dout, apart.transpose(0, 1), k, v, *want, seg)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    pad = torch.zeros(n, h, d + 4, dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError):
        spc.spc_attention_fwd(q, k, v, seg, out=pad[:, :, :d])
    with pytest.raises(ValueError):
        spc.spc_attention_bwd(dout, q, k, v, *want, seg, dq=torch.empty_like(q).float())


@pytest.mark.parametrize("skip", [1, 4, 8])
def test_attention_of_tensors_that_start_anywhere(skip):
    """Off a 16-byte boundary the CUDA cores take the call."""
    q, k, v, dout, seg, _ = attn_case(2, 2, 32, [90, 40], None, 0, "bf16")
    moved = []
    for t in (q, k, v, dout):
        flat = torch.zeros(t.numel() + skip, dtype=t.dtype, device=dev())
        flat[skip:] = to(t).view(-1)
        moved.append(flat[skip:].view(t.shape))
    o, lse = spc.spc_attention_fwd(*moved[:3], offsets(*seg))
    grads = spc.spc_attention_bwd(moved[3], *moved[:3], o, lse, offsets(*seg))
    check_attention(q, k, v, dout, seg, seg, "bf16", (o, lse, grads))


def test_attention_rows_with_gaps():
    """Row strides that are no multiple of 16 bytes, and rows with room between them."""
    g = gen(8)
    for gap, dtype in ((3, "bf16"), (8, "f16"), (5, "f32")):
        n, h, d = 130, 2, 40
        wide = normal(g, n, 3 * h * d + gap, dtype=dtype)
        t = to(wide)
        q, k, v = (t.as_strided((n, h, d), (t.stride(0), d, 1), i * h * d) for i in range(3))
        cpu = [wide[:, i * h * d:(i + 1) * h * d].reshape(n, h, d) for i in range(3)]
        dout = normal(g, n, h, d, dtype=dtype)
        o, lse = spc.spc_attention_fwd(q, k, v, offsets(0, 30, 130))
        grads = spc.spc_attention_bwd(to(dout), q, k, v, o, lse, offsets(0, 30, 130))
        check_attention(*cpu, dout, [0, 30, 130], [0, 30, 130], dtype, (o, lse, grads))


def test_outputs_given_by_the_caller_are_used():
    g = gen(9)
    x, q = normal(g, 40, 24).to(dev()), normal(g, 40, 2, 16, dtype="bf16").to(dev())
    y, mean, rstd = torch.empty_like(x), torch.empty(40, device=dev()), torch.empty(40, device=dev())
    got = spc.spc_layer_norm_fwd(x, None, None, out=y, mean=mean, rstd=rstd)
    assert [t.data_ptr() for t in got] == [t.data_ptr() for t in (y, mean, rstd)]
    dg, db, ws = torch.empty(24, device=dev()), torch.empty(24, device=dev()), torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    got = spc.spc_layer_norm_bwd(x, x, None, mean, rstd, dgamma=dg, dbeta=db, ws=ws)
    assert got[1].data_ptr() == dg.data_ptr() and got[2].data_ptr() == db.data_ptr()
    e, w = torch.empty(40, 3, dtype=torch.int32, device=dev()), torch.empty(40, 3, device=dev())
    got = spc.spc_route_fwd(x, 3, expert=e, gate=w)
    assert got[0].data_ptr() == e.data_ptr() and got[1].data_ptr() == w.data_ptr()
    for bad in (torch.empty(40, 3, device=dev()), torch.empty(41, 3, dtype=torch.int32, device=dev())):
        with pytest.raises(ValueError):
            spc.spc_route_fwd(x, 3, expert=bad)
    with pytest.raises(ValueError):
        spc.spc_attention_fwd(q, q, q, offsets(0, 40), lse=torch.empty(40, 3, device=dev()))
    with pytest.raises(ValueError):
        spc.spc_attention_fwd(q, q[:30], q[:30], offsets(0, 40))  # as many keys as queries, or offsets of their own
    with pytest.raises(ValueError):
        spc.spc_attention_fwd(q, q, q, offsets(0, 40), status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        spc.spc_rope_fwd(q, torch.zeros(40, 4, dtype=torch.int64, device=dev()), spc.spc_rope_steps((1, 1, 1)), (1, 1, 1))
    with pytest.raises(ValueError):
        spc.spc_rope_fwd(q, torch.zeros(40, 4, dtype=torch.int32, device=dev()), spc.spc_rope_steps((1, 1, 2)), (1, 1, 1))
    with pytest.raises(spc.SpcError):
        spc.spc_attention_bwd(q, q, q, q, q, torch.zeros(40, 2, device=dev()), offsets(0, 40), dq=q)


# ------------------------------------------------------------------ streams
def test_calls_on_two_streams_at_once():
    """Two streams with workspaces of their own: results are those of each call alone."""
    cases = [attn_case(4, 2, 64, [600, 300], None, 0, "bf16", seed=s) for s in range(2)]
    seg = offsets(0, 600, 900)
    args = [[t.to(dev()) for t in c[:4]] for c in cases]

    def both(q, k, v, dout):
        o, lse = spc.spc_attention_fwd(q, k, v, seg)
        return [o, lse, *spc.spc_attention_bwd(dout, q, k, v, o, lse, seg)]

    want = [both(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = both(*args[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_graphs_share_a_workspace():
    """Split calls of two graphs that run one after the other with the same workspace."""
    cases = [attn_case(2, 2, 64, [3], [5000 + 700 * s], 0, "f16", seed=s) for s in range(2)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=dev())
    graphs, held, want = [], [], []
    for q, k, v, dout, seg, seg_k in cases:
        a = [to(t) for t in (q, k, v)]
        g, s, sk = to(dout), offsets(*seg), offsets(*seg_k)

        def call():
            o, lse = spc.spc_attention_fwd(*a, s, seg_k=sk, ws=ws)
            return [o, lse, *spc.spc_attention_bwd(g, *a, o, lse, s, seg_k=sk, ws=ws)]

        want.append([t.clone() for t in call()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(call())
        graphs.append((graph, a, g, s, sk))
    for _ in range(2):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ differences
def slope(f, x, direction, h):
    """The derivative of f along a direction by the fourth-order central difference, f summed in float64."""
    def at(t):
        return float(f((x.double() + t * direction.double()).float().to(dev())))

    return (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)


def test_gradients_are_the_slopes_of_the_forward_calls():
    """fp32, h = 2^-6: the difference is off by h^4 / 30 of a fifth derivative (functions of order 1) and by rounding, about
    2^-24 sqrt(n) |f's terms| / h; a hundredth of the slope's size bounds both."""
    g = gen(12)
    h = 2.0 ** -6

    def check(f, x, grad):
        for _ in range(3):
            direction = normal(g, *x.shape)
            direction /= direction.norm() / math.sqrt(direction.numel()) * 4
            want = float((grad.double().cpu() * direction.double()).sum())
            got = slope(f, x, direction, h)
            assert abs(got - want) <= 0.01 * float(grad.double().norm().cpu() * direction.double().norm()), (got, want)

    x, ga, be, dy = normal(g, 40, 24), normal(g, 24), normal(g, 24), normal(g, 40, 24)
    y, mean, rstd = spc.spc_layer_norm_fwd(to(x), to(ga), to(be))
    dx, dgamma, dbeta = spc.spc_layer_norm_bwd(to(dy), to(x), to(ga), mean, rstd)
    weigh = lambda t, w: (t.double() * w.to(dev()).double()).sum()  # noqa: E731
    check(lambda t: weigh(spc.spc_layer_norm_fwd(t, to(ga), to(be))[0], dy), x, dx)
    check(lambda t: weigh(spc.spc_layer_norm_fwd(to(x), t, to(be))[0], dy), ga, dgamma)
    check(lambda t: weigh(spc.spc_layer_norm_fwd(to(x), to(ga), t)[0], dy), be, dbeta)
    coords = torch.randint(-40, 40, (40, 4), generator=g, dtype=torch.int32)
    steps, heads, dh = spc.spc_rope_steps((3, 2, 1)), normal(g, 40, 2, 13), normal(g, 40, 2, 13)
    check(lambda t: weigh(spc.spc_rope_fwd(t, to(coords), steps, (3, 2, 1)), dh), heads, spc.spc_rope_bwd(to(dh), to(coords), steps, (3, 2, 1)))
    for score in (0, 1):
        for renorm in (True, False):
            # experts well apart, so that no step changes the choice
            logits = torch.stack([torch.randperm(12, generator=g) for _ in range(30)]).float()
            dgate = normal(g, 30, 4)
            expert, _ = spc.spc_route_fwd(to(logits), 4, score=score, renorm=renorm)
            dl = spc.spc_route_bwd(to(dgate), to(logits), expert, score=score, renorm=renorm)
            check(lambda t: weigh(spc.spc_route_fwd(t, 4, score=score, renorm=renorm)[1], dgate), logits, dl)
    q, k, v, dout, seg, seg_k = attn_case(4, 2, 16, [30, 70], [50, 41], 0, "f32", std=1.0)
    s, sk = offsets(*seg), offsets(*seg_k)
    o, lse = spc.spc_attention_fwd(to(q), to(k), to(v), s, seg_k=sk)
    dq, dk, dv = spc.spc_attention_bwd(to(dout), to(q), to(k), to(v), o, lse, s, seg_k=sk)
    check(lambda t: weigh(spc.spc_attention_fwd(t, to(k), to(v), s, seg_k=sk)[0], dout), q, dq)
    check(lambda t: weigh(spc.spc_attention_fwd(to(q), t, to(v), s, seg_k=sk)[0], dout), k, dk)
    check(lambda t: weigh(spc.spc_attention_fwd(to(q), to(k), t, s, seg_k=sk)[0], dout), v, dv)


# ------------------------------------------------------------------ shapes at the kernels' borders
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,sizes_q,sizes_k", [
    (1, 1, 64, [128], [64]), (1, 1, 64, [256], [128]), (1, 1, 128, [257], [65]), (2, 2, 64, [19000], [70]), (8, 8, 128, [5000], [200]),
    (8, 2, 128, [2500, 2600], [90, 300]), (24, 1, 64, [900, 17], [333, 64]), (128, 1, 16, [5, 4], [70, 3]), (130, 1, 8, [3], [100]),
    (67, 67, 8, [9], [200]), (2, 1, 64, [64, 65, 63, 1], [1, 64, 65, 63]), (6, 6, 56, [2049], [2049])])
def test_attention_at_tile_borders(hq, hk, d, sizes_q, sizes_k, dtype):
    case = attn_case(hq, hk, d, sizes_q, sizes_k, 0, dtype)
    check_attention(*case, dtype, run_attention(*case, dtype))


@pytest.mark.parametrize("hq,hk,d,sizes_q,sizes_k,outside", [
    (1, 1, 16, [128], [128], 0), (2, 1, 12, [129, 1, 300], [257, 0, 131], 2), (3, 3, 4, [127], [1], 0), (4, 4, 8, [20], [5000], 0),
    (4, 2, 16, [1500], [1500], 3), (1, 1, 16, [5, 4, 3], [33, 129, 4], 0), (2, 2, 16, [40] * 30, None, 0), (6, 2, 16, [1], [100], 1)])
def test_attention_of_narrow_heads(hq, hk, d, sizes_q, sizes_k, outside):
    case = attn_case(hq, hk, d, sizes_q, sizes_k, outside, "f32")
    check_attention(*case, "f32", run_attention(*case, "f32"))


def test_attention_of_narrow_heads_with_bad_values():
    """NaN and infinities stay in their segment and their row, and keys that score -inf have no part."""
    q, k, v, dout, seg, _ = attn_case(2, 2, 16, [140, 150, 60], None, 0, "f32")
    o, lse = spc.spc_attention_fwd(to(q), to(k), to(v), offsets(*seg))
    q[3, 0, 5] = math.nan
    k[200, 1, 2], v[201, 0] = math.nan, math.inf
    k[300, :], q[290:, :] = -math.inf, q[290:, :].abs() + 0.1  # no query of the last segment scores it
    o2, lse2 = spc.spc_attention_fwd(to(q), to(k), to(v), offsets(*seg))
    bad = torch.zeros(350, 2, dtype=torch.bool)
    bad[3, 0] = bad[140:290, 1] = True
    assert torch.equal(lse2.isnan().cpu(), bad)
    assert not o2[bad.to(o2.device)].isfinite().any() and not o2[140:290, 0].isfinite().any()
    same = ~bad
    same[140:290, 0] = same[290:] = False
    assert torch.equal(o2[same.to(o2.device)], o[same.to(o2.device)]) and torch.equal(lse2[:140][same[:140].to(o2.device)], lse[:140][same[:140].to(o2.device)])
    keep = [i for i in range(290, 350) if i != 300]
    want, _ = spc.spc_attention_fwd(to(q[290:]), to(k[keep]), to(v[keep]), offsets(0, 60), seg_k=offsets(0, 59))
    assert torch.allclose(o2[290:], want, rtol=1e-5, atol=1e-5)
    all_out = torch.full((70, 2, 16), -math.inf)
    o3, lse3 = spc.spc_attention_fwd(to(q[290:]), to(all_out), to(v[:70]), offsets(0, 60), seg_k=offsets(0, 70))
    assert not o3.any() and bool((lse3 == -math.inf).all())


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_attention_scales(scale):
    for dtype in ("f32", "bf16"):
        case = attn_case(2, 2, 24, [120, 90], None, 0, dtype, std=0.7)
        check_attention(*case, dtype, run_attention(*case, dtype, scale), scale)
