"""The layers between convolutions where a kernel changes its way: the last bit of dropout at either
alignment, parts of a segment that one row fills, the tiles of CTA pairs and of long rows, empty lists,
keys and row lists of wider types, views off a 16-byte boundary, very long rows.

Bounds are those of test_gpu_layers.py where nothing else is said."""

import ctypes

import numpy as np
import pytest
import torch

import layers_ref as ref
import sparse_convolution_hash_gb300 as spc
from gpu_util import DT, dev
from sparse_convolution_hash_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def to_dev(a):
    if a is None:
        return None
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).to(dev())


def close(got, want, bound, what=""):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, worst {((got - want).abs() - bound).max():.3g}"


# --------------------------------------------------------------------- dropout
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,skip", [(40003, 0), (40003, 1)])
def test_dropout_is_a_product_and_a_sum_in_fp32(n, skip, dtype, residual):
    """Every element has the bits of x s in fp32, s = 1 / (1 - p) in fp32, plus the residual in fp32,
    rounded to the type: in whole vectors, in the last partial one and off a 16-byte boundary."""
    g = np.random.default_rng(n + skip)
    x = to_dev(torch.from_numpy(g.standard_normal(n + skip)).to(DT[dtype]))[skip:]
    res = to_dev(torch.from_numpy(g.standard_normal(n + skip)).to(DT[dtype]))[skip:]
    p, seed, offset = 0.1, 0x1234567890ABCDEF, 7
    y = spc.spc_dropout_fwd(x, p, to_dev(torch.tensor([seed, offset])), residual=res if residual else None)
    keep = torch.from_numpy(ref.dropout_words(seed, offset, 0, n) >= np.uint64(round(p * 2 ** 32)))
    want = torch.where(keep, x.cpu().float() * torch.tensor(1 / (1 - p), dtype=torch.float32), torch.zeros(()))
    if residual:
        want = want + res.cpu().float()
    assert torch.equal(y.cpu(), want.to(DT[dtype]))


# ------------------------------------------------------------------ group norm
def share_rows(n):
    """Positions that one CTA of the group norm owns: one CTA for each SM, 64 positions at least."""
    shares = max(1, min(torch.cuda.get_device_properties(dev()).multi_processor_count, -(-n // 64)))
    return -(-n // shares)


@pytest.mark.parametrize("first", [0.0, 1100.0])
@pytest.mark.parametrize("n", [40000, 498145])
def test_group_norm_segment_that_starts_on_a_last_position(n, first):
    """The first part of the second segment is one row, far from the others at 1000 +- 1: the parts
    join without losing the variance's digits."""
    g = np.random.default_rng(0)
    x = torch.from_numpy(1000 + g.standard_normal((n, 16))).float()
    cut = share_rows(n) - 1
    x[cut] = first
    seg = np.array([0, cut, n], np.int32)
    y_r, mean_r, rstd_r, _ = ref.norm_fwd(x, None, None, seg, None, 4, 1e-5, "none")
    y, mean, rstd = spc.spc_group_norm_fwd(to_dev(x), None, None, to_dev(seg), 4)
    # as for one segment with such a first row: the values' distances from the mean are exact to
    # 1000 e / spread and 1e-4 covers that and the sums around pivots
    assert float((rstd.double().cpu() / rstd_r - 1).abs().max()) < 1e-4
    assert float((mean.double().cpu() / mean_r - 1).abs().max()) < 1e-6
    assert float((y.double().cpu() - y_r).norm() / y_r.norm()) < 1e-3


# ------------------------------------------------------------- grouped products
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cin,cout", [(64, 64), (256, 256), (33, 40)])
def test_grouped_weight_gradient_of_no_positions(cin, cout, dtype):
    """m = 0 with row lists (which are not NULL) and operands that have rows: dW is zeros."""
    d, L = dev(), binding.lib()
    x, dy = torch.randn(7, cin, device=d).to(DT[dtype]), torch.randn(5, cout, device=d).to(DT[dtype])
    rows = torch.zeros(8, dtype=torch.int32, device=d)
    seg = torch.zeros(4, dtype=torch.int32, device=d)
    dw = torch.full((3, cin, cout), 7.0, device=d)
    dt = {"f32": 0, "f16": 1, "bf16": 2}[dtype]
    need = L.spc_grouped_workspace_size(3, 0, cin, cout, dt, 1)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=d)
    st = spc.new_status(d)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    code = L.spc_grouped_wgrad(p(x), p(dy), p(seg), p(rows), p(rows), 3, 7, 5, 0, cin, cout, dt, p(dw), p(st), p(ws),
                               ws.numel(), ctypes.c_void_p(torch.cuda.current_stream(d).cuda_stream))
    assert code == 0, binding.spc_status_string(code)
    spc.check_status(st)
    assert float(dw.abs().max()) == 0


# ----------------------------------------------- keys and row lists of other types
def test_keys_and_lists_of_wider_types_keep_their_values():
    """A key or row number that 32 bits do not hold is out of range, not its low half."""
    d = dev()
    wide = torch.tensor([2 ** 32, 1, -1, 2 ** 32 + 1, 0, 2 ** 31, 1 - 2 ** 32, -2 ** 63, 2 ** 63 - 1], device=d)
    seg, order = spc.spc_row_segments(wide, 2)
    assert seg.tolist() == [0, 1, 2] and order.tolist() == [4, 1, 0, 2, 3, 5, 6, 7, 8]
    for dt in (torch.uint8, torch.int16, torch.int64, torch.uint32, torch.uint64):
        seg, order = spc.spc_row_segments(torch.tensor([1, 0, 2, 1], device=d).to(dt), 2)
        assert seg.tolist() == [0, 1, 3] and order.tolist() == [1, 0, 3, 2]
    high = torch.tensor([1, -2], device=d).view(torch.uint64)  # 2^64 - 2
    assert spc.spc_row_segments(high, 2)[0].tolist() == [0, 0, 1]
    x = torch.randn(6, 16, device=d)
    w = torch.randn(1, 16, 8, device=d)
    seg = torch.tensor([0, 6], device=d)  # offsets of 64 bits are read as they are
    rows = torch.arange(6, device=d)
    want = spc.spc_grouped_fwd(x, w, seg)
    assert torch.equal(spc.spc_grouped_fwd(x, w, seg, x_rows=rows, y_rows=rows), want)
    rows[3] = 2 ** 32 + 3
    for f in (lambda st: spc.spc_grouped_fwd(x, w, seg, x_rows=rows, status=st),
              lambda st: spc.spc_grouped_wgrad(x, want, seg, y_rows=rows, status=st),
              lambda st: spc.spc_group_norm_fwd(x, None, None, seg, 4, order=rows, status=st),
              lambda st: spc.spc_grouped_fwd(x, w, torch.tensor([0, 2 ** 32 + 6], device=d), status=st)):
        st = spc.new_status(d)
        f(st)
        assert int(st) == 10


def test_keys_and_lists_are_whole_numbers():
    d = dev()
    x = torch.randn(6, 16, device=d)
    w = torch.randn(1, 16, 8, device=d)
    seg = torch.tensor([0, 6], dtype=torch.int32, device=d)
    for f in (lambda: spc.spc_row_segments(torch.tensor([0.5, 1.0], device=d), 2),
              lambda: spc.spc_grouped_fwd(x, w, seg.float()),
              lambda: spc.spc_grouped_fwd(x, w, seg, x_rows=torch.zeros(6, device=d)),
              lambda: spc.spc_group_norm_fwd(x, None, None, seg, 4, order=torch.zeros(6, device=d))):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------ views off a 16-byte boundary
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cin,cout", [(33, 65), (36, 20), (33, 8), (8, 33)])
def test_grouped_products_of_rows_that_start_anywhere(cin, cout, dtype):
    """Slices of the first axis start on their rows' own boundary: odd rows on an element's, rows of a
    multiple of four on four elements'.  The products are those of aligned copies."""
    g = torch.Generator().manual_seed(cin + cout)
    mk = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).to(dev())[1:]
    x, dy, w = mk(301, cin), mk(301, cout), mk(4, cin, cout)
    seg = to_dev(np.array([0, 100, 100, 290], np.int32))
    y = torch.empty(301, cout, device=dev(), dtype=DT[dtype])[1:]
    dx = torch.empty(301, cin, device=dev(), dtype=DT[dtype])[1:]
    dw = torch.empty(4, cin, cout, device=dev())[1:]
    c = lambda t: t.clone()
    assert torch.equal(spc.spc_grouped_fwd(x, w, seg, out=y), spc.spc_grouped_fwd(c(x), c(w), seg))
    assert torch.equal(spc.spc_grouped_dgrad(dy, w, seg, out=dx), spc.spc_grouped_dgrad(c(dy), c(w), seg))
    assert torch.equal(spc.spc_grouped_wgrad(x, dy, seg, out=dw), spc.spc_grouped_wgrad(c(x), c(dy), seg))


# ------------------------------------------------------------- very long rows
@pytest.mark.parametrize("c,groups", [(1026, 2), (1026, 513)])
def test_group_norm_of_very_long_rows_far_from_zero(c, groups):
    """Rows of more than 512 vectors at 1000.3 +- 0.01: a sum of the values themselves would take the
    same side at every rounding and move the mean by many spreads."""
    n = 20000
    g = np.random.default_rng(2)
    x = torch.from_numpy(1000.3 + 0.01 * g.standard_normal((n, c))).float()
    seg = np.array([0, n - 700, n], np.int32)
    _, mean_r, rstd_r, _ = ref.norm_fwd(x, None, None, seg, None, groups, 1e-12, "none")
    y, mean, rstd = spc.spc_group_norm_fwd(to_dev(x), None, None, to_dev(seg), groups, eps=1e-12)
    # the mean is rounded to fp32 (2^-24 relative, 6e-5 here) after sums around a pivot that lose
    # less than as much again; squares around it are off by (1e-4 / 0.01)^2 of the variance
    assert float((mean.double().cpu() / mean_r - 1).abs().max()) < 2 * ref.EPS32
    assert float((rstd.double().cpu() / rstd_r - 1).abs().max()) < 2e-4
    y_r = ((x.double() - mean.double().cpu().repeat_interleave(c // groups, 1)[(torch.arange(n) >= n - 700).long()])
           * rstd_r.repeat_interleave(c // groups, 1)[(torch.arange(n) >= n - 700).long()])
    assert float((y.double().cpu() - y_r).norm() / y_r.norm()) < 1e-3


# ------------------------------------------------------- where buffers have to be
def test_status_words_and_workspaces_are_on_the_device():
    d = dev()
    x = torch.randn(10, 16, device=d)
    seg = torch.tensor([0, 10], dtype=torch.int32, device=d)
    w = torch.randn(1, 16, 8, device=d)
    dy = torch.randn(10, 8, device=d)
    m = torch.zeros(1, 4, device=d)
    host, host_ws = torch.zeros(1, dtype=torch.int32), torch.empty(1 << 20, dtype=torch.uint8)
    calls = [lambda **k: spc.spc_group_norm_fwd(x, None, None, seg, 4, **k),
             lambda **k: spc.spc_group_norm_bwd(x, x, None, None, m, m + 1, seg, 4, **k),
             lambda **k: spc.spc_grouped_fwd(x, w, seg, **k), lambda **k: spc.spc_grouped_dgrad(dy, w, seg, **k),
             lambda **k: spc.spc_grouped_wgrad(x, dy, seg, **k)]
    for f in calls:
        for bad in (host, torch.zeros(1, device=d), torch.zeros(0, dtype=torch.int32, device=d)):
            with pytest.raises(ValueError):
                f(status=bad)
        for bad in (host_ws, torch.zeros(1, dtype=torch.uint8, device=d).expand(1 << 20)):
            with pytest.raises(ValueError):
                f(ws=bad)
    with pytest.raises(ValueError):
        spc.spc_row_segments(seg, 2, ws=host_ws)


# ---------------------------------------------------- tiles that long segments take
def ragged(segments, m, x_rows, y_rows, dtype, cin, cout, seed=0):
    g = np.random.default_rng(seed + m + cin + cout)
    x = torch.from_numpy(g.standard_normal((m, cin))).to(DT[dtype])
    dy = torch.from_numpy(g.standard_normal((m, cout))).to(DT[dtype])
    w = torch.from_numpy(g.standard_normal((segments, cin, cout)) / np.sqrt(cin)).to(DT[dtype])
    perm = lambda: g.permutation(m).astype(np.int32)
    return x, dy, w, perm() if x_rows else None, perm() if y_rows else None


def check_products(x, dy, w, seg, x_rows, y_rows, dtype, wgrad=False):
    """Forward, gradient by the input and (on request) by the weights against float64, twice the same."""
    m, cin, cout = x.shape[0], x.shape[1], dy.shape[1]
    u, st = ref.U[DT[dtype]], spc.new_status(dev())
    lists = dict(x_rows=to_dev(x_rows), y_rows=to_dev(y_rows), status=st)
    f = lambda: spc.spc_grouped_fwd(to_dev(x), to_dev(w), to_dev(seg), **lists)
    y = f()
    want, mag = ref.grouped_fwd(x, w, seg, x_rows, y_rows, m)
    close(y, want, 1.01 * u * want.abs() + cin * 2.0 ** -23 * mag * 1.01 + 2.0 ** -25 * (mag > 0), "y")
    assert torch.equal(y, f())
    f = lambda: spc.spc_grouped_dgrad(to_dev(dy), to_dev(w), to_dev(seg), **lists)
    dx = f()
    want, mag = ref.grouped_fwd(dy, w.transpose(1, 2), seg, y_rows, x_rows, m)
    close(dx, want, 1.01 * u * want.abs() + cout * 2.0 ** -23 * mag * 1.01 + 2.0 ** -25 * (mag > 0), "dx")
    assert torch.equal(dx, f())
    if wgrad:
        f = lambda: spc.spc_grouped_wgrad(to_dev(x), to_dev(dy), to_dev(seg), **lists)
        dw = f()
        want, mag = ref.grouped_wgrad(x, dy, seg, x_rows, y_rows)
        close(dw, want, torch.from_numpy(np.diff(seg).astype(np.float64))[:, None, None] * 2.0 ** -23 * mag, "dw")
        assert torch.equal(dw, f())
    spc.check_status(st)


# offsets with rows of no segment on both sides, an empty segment, one shorter than a CTA's 128 rows
# (the second CTA of a pair has none), and a last tile of 74 rows
LONG = np.array([40, 6000, 6000, 6100, 8990], np.int32)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,cin,cout,seg", [
    (9000, 520, 520, LONG),                                              # pairs both ways, columns 520 = 2 x 256 + 8
    (10500, 512, 264, np.array([0, 5000, 10500], np.int32)),             # pairs forward; dgrad: K of 264, no pairs
    (10500, 264, 512, np.array([3, 4100, 4101, 4101, 10499], np.int32)),  # pairs in dgrad; a segment of one row
    (12800, 1024, 512, np.array([0, 2560, 5120, 7680, 10240, 12800], np.int32))])  # whole tiles, deep K
def test_grouped_products_of_long_dense_segments(m, cin, cout, seg, dtype):
    check_products(*ragged(len(seg) - 1, m, False, False, dtype, cin, cout)[:3], seg, None, None, dtype, wgrad=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cin,cout", [(520, 520), (264, 1024)])
def test_grouped_products_of_long_listed_segments(cin, cout, dtype):
    """128 x 256 tiles with rows through lists, forward and gradient by the input."""
    x, dy, w, xr, yr = ragged(4, 9000, True, True, dtype, cin, cout)
    check_products(x, dy, w, LONG, xr, yr, dtype, wgrad=True)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("cin,cout", [(33, 385), (36, 388)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_products_in_large_cuda_core_tiles(dtype, cin, cout, listed):
    """128 x 128 tiles on CUDA cores (two for each SM), values one by one and four at a time."""
    m, seg = 26000, np.array([5, 9000, 9000, 9100, 25999], np.int32)
    x, dy, w, xr, yr = ragged(4, m, listed, listed, dtype, cin, cout)
    st = spc.new_status(dev())
    y = spc.spc_grouped_fwd(to_dev(x), to_dev(w), to_dev(seg), x_rows=to_dev(xr), y_rows=to_dev(yr), status=st)
    want, mag = ref.grouped_fwd(x, w, seg, xr, yr, m)
    u = ref.U[DT[dtype]]
    close(y, want, 1.01 * u * want.abs() + cin * 2.0 ** -23 * mag * 1.01 + 2.0 ** -25 * (mag > 0), "y")
    # the gradient by the input of the mirrored shape has as many columns
    x, dy, w, xr, yr = ragged(4, m, listed, listed, dtype, cout, cin)
    dx = spc.spc_grouped_dgrad(to_dev(dy), to_dev(w), to_dev(seg), x_rows=to_dev(xr), y_rows=to_dev(yr), status=st)
    want, mag = ref.grouped_fwd(dy, w.transpose(1, 2), seg, yr, xr, m)
    close(dx, want, 1.01 * u * want.abs() + cin * 2.0 ** -23 * mag * 1.01 + 2.0 ** -25 * (mag > 0), "dx")
    spc.check_status(st)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("cin,cout", [(129, 257), (132, 260)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_grouped_weight_gradient_in_large_cuda_core_tiles(dtype, cin, cout, listed):
    segments, m = 52, 900
    g = np.random.default_rng(cin)
    seg = np.sort(g.integers(0, m + 1, segments + 1)).astype(np.int32)
    x, dy, w, xr, yr = ragged(segments, m, listed, listed, dtype, cin, cout)
    check_products(x, dy, w, seg, xr, yr, dtype, wgrad=True)


def test_wait_limit_ends_products_of_long_segments_with_a_status():
    """As for the other shapes: with a limit of 0 the pair kernels give up, report it and return, and
    the same calls work again afterwards."""
    d = dev()
    x = torch.randn(9000, 520, device=d, dtype=torch.bfloat16)
    w = torch.randn(4, 520, 520, device=d, dtype=torch.bfloat16)
    seg, rows = to_dev(LONG), torch.randperm(9000, device=d).to(torch.int32)
    calls = [lambda st: spc.spc_grouped_fwd(x, w, seg, status=st), lambda st: spc.spc_grouped_dgrad(x, w, seg, status=st),
             lambda st: spc.spc_grouped_dgrad(x, w, seg, y_rows=rows, status=st),
             lambda st: spc.spc_grouped_wgrad(x, x, seg, status=st),
             lambda st: spc.spc_grouped_wgrad(x, x, seg, x_rows=rows, y_rows=rows, status=st)]
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
