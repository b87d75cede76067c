"""The float64 forms that the GPU layers are compared with, held to independent
facts on the CPU: torch's own group norm, central differences, the published
known answers of Philox4x32-10, and the C entry points' argument checks."""

import ctypes

import numpy as np
import pytest
import torch

import layers_ref as ref
from sparse_convolution_hash_gb300 import binding
from sparse_convolution_hash_gb300 import build as libbuild


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return binding.lib()


@pytest.mark.parametrize("kind", ["none", "relu", "silu"])
def test_norm_forward_is_torch_group_norm_per_sample(kind):
    torch.manual_seed(0)
    x = torch.randn(37, 24, dtype=torch.float64) * 3 + 2
    gamma, beta = torch.randn(24, dtype=torch.float64), torch.randn(24, dtype=torch.float64)
    seg = np.array([0, 20, 20, 37], np.int32)
    y, mean, rstd, _ = ref.norm_fwd(x, gamma, beta, seg, None, 6, 1e-5, kind)
    for lo, hi in ((0, 20), (20, 37)):
        z = torch.nn.functional.group_norm(x[lo:hi].T[None], 6, gamma, beta, 1e-5)[0].T
        z = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu}[kind](z)
        assert torch.allclose(y[lo:hi], z, rtol=1e-12, atol=1e-12)
    assert mean[1].abs().max() == 0 and torch.allclose(rstd[1], torch.full((6,), 1e-5, dtype=torch.float64) ** -0.5)


@pytest.mark.parametrize("kind", ["none", "silu"])
def test_norm_backward_is_the_central_difference(kind):
    torch.manual_seed(1)
    seg, order = np.array([0, 5, 12, 13], np.int32), np.random.default_rng(0).permutation(14).astype(np.int32)
    x, dy = torch.randn(14, 6, dtype=torch.float64), torch.randn(14, 6, dtype=torch.float64)
    gamma, beta = torch.randn(6, dtype=torch.float64), torch.randn(6, dtype=torch.float64)

    def loss(x, gamma, beta):
        return float((dy * ref.norm_fwd(x, gamma, beta, seg, order, 3, 1e-5, kind)[0]).sum())

    _, mean, rstd, _ = ref.norm_fwd(x, gamma, beta, seg, order, 3, 1e-5, kind)
    got = ref.norm_bwd(dy, x, gamma, beta, mean, rstd, seg, order, 3, kind)
    h = 1e-5
    for k, (arg, grad) in enumerate(zip((x, gamma, beta), got)):
        for _ in range(6):
            v = torch.randn_like(arg)
            plus, minus = [x, gamma, beta], [x, gamma, beta]
            plus[k], minus[k] = arg + h * v, arg - h * v
            want = (loss(*plus) - loss(*minus)) / (2 * h)
            # error of a central difference: h^2 f''' / 6 and rounding 1e-16 f / h
            assert abs(want - float((grad * v).sum())) < 1e-6 * (1 + abs(want))


def test_philox_known_answers():
    f = 0xFFFFFFFF
    assert ref.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_segments_form():
    seg, order = ref.segments(np.array([2, 0, -1, 2, 7, 0]), 3)
    assert seg.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 5, 0, 3, 2, 4]


P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = 1, 6, 8


def test_status_of_a_bad_row_index_has_a_name(L):
    assert binding.spc_status_string(10) == "segment offset or row index out of range"
    assert binding.STATUS_NAMES[10] == "SPC_ERR_ROW_INDEX"


def test_row_segments_refusals(L):
    def f(ids=P(256), stride=1, n=4, s=2, seg=P(256), order=P(256), ws=P(256), nb=1 << 20):
        return L.spc_row_segments(ids, stride, n, s, seg, order, ws, nb, None)

    assert f(n=-1) == INVALID and f(s=0) == INVALID and f(s=1025) == INVALID
    assert f(stride=0) == INVALID and f(ids=None) == INVALID and f(seg=None) == INVALID
    assert f(ids=P(258)) == INVALID and f(order=P(257)) == INVALID
    assert f(n=2 ** 31) == UNSUPPORTED and f(stride=2 ** 62) == UNSUPPORTED
    assert f(ws=None) == WORKSPACE and f(nb=4) == WORKSPACE
    assert L.spc_row_segments_workspace_size(-1, 2) == 0
    assert L.spc_row_segments_workspace_size(5, 1025) == 0
    assert L.spc_row_segments_workspace_size(0, 1) > 0


def test_group_norm_refusals(L):
    def fwd(x=P(256), gamma=P(256), seg=P(256), order=None, s=2, n=4, c=8, g=2, eps=1e-5, act=0, dt=0,
            y=P(256), mean=P(256), rstd=P(256), ws=P(256), nb=1 << 30):
        return L.spc_group_norm_fwd(x, gamma, None, seg, order, s, n, c, g, eps, act, dt, y, mean, rstd,
                                    None, ws, nb, None)

    def bwd(dy=P(256), x=P(256), seg=P(256), s=2, n=4, c=8, g=2, act=0, dt=0, dx=P(256), mean=P(256),
            dgamma=None, ws=P(256), nb=1 << 30):
        return L.spc_group_norm_bwd(dy, x, None, None, mean, P(256), seg, None, s, n, c, g, act, dt, dx,
                                    dgamma, None, None, ws, nb, None)

    assert fwd(n=-1) == INVALID and fwd(c=0) == INVALID and fwd(g=0) == INVALID and fwd(g=3) == INVALID
    assert fwd(s=0) == INVALID and fwd(s=5000) == INVALID and fwd(act=3) == INVALID and fwd(dt=3) == INVALID
    assert fwd(eps=0.0) == INVALID and fwd(eps=float("nan")) == INVALID and fwd(eps=float("inf")) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID and fwd(seg=None) == INVALID
    assert fwd(mean=None) == INVALID and fwd(rstd=None) == INVALID
    assert fwd(x=P(257)) == INVALID and fwd(x=P(258)) == INVALID and fwd(order=P(258)) == INVALID
    assert fwd(n=2 ** 31) == UNSUPPORTED
    assert fwd(ws=None) == WORKSPACE and fwd(nb=0) == WORKSPACE and fwd(ws=P(128)) == WORKSPACE
    assert bwd(dy=None) == INVALID and bwd(x=None) == INVALID and bwd(dx=None) == INVALID
    assert bwd(g=5) == INVALID and bwd(act=-1) == INVALID and bwd(mean=None) == INVALID
    assert bwd(dgamma=P(258)) == INVALID and bwd(dy=P(258)) == INVALID
    assert bwd(nb=0) == WORKSPACE
    assert L.spc_group_norm_workspace_size(10, 8, 2, 3, 0) == 0


def test_dropout_refusals(L):
    def fwd(x=P(256), res=None, n=4, p=0.5, rng=P(256), dt=0, y=P(256)):
        return L.spc_dropout_fwd(x, res, n, p, rng, dt, y, None)

    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert fwd(p=p) == INVALID
    assert fwd(n=-1) == INVALID and fwd(dt=5) == INVALID and fwd(rng=None) == INVALID and fwd(rng=P(260)) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID and fwd(x=P(258)) == INVALID and fwd(res=P(258)) == INVALID
    assert fwd(n=0, x=None, y=None) == 0
    assert L.spc_dropout_bwd(None, 4, 0.5, P(256), 0, P(256), None) == INVALID
    assert L.spc_dropout_bwd(P(256), 4, 2.0, P(256), 0, P(256), None) == INVALID


def test_grouped_refusals(L):
    def fwd(x=P(256), w=P(256), seg=P(256), xr=None, yr=None, s=2, n=4, m=4, ci=8, co=8, dt=0, y=P(256),
            f=L.spc_grouped_fwd):
        return f(x, w, seg, xr, yr, s, n, m, ci, co, dt, y, None, P(256), 1 << 40, None)

    for f in (L.spc_grouped_fwd, L.spc_grouped_dgrad):
        assert fwd(f=f, x=None) == INVALID and fwd(f=f, w=None) == INVALID and fwd(f=f, y=None) == INVALID
        assert fwd(f=f, seg=None) == INVALID and fwd(f=f, x=P(264)) == INVALID and fwd(f=f, w=P(264)) == INVALID
        assert fwd(f=f, m=-1) == INVALID and fwd(f=f, n=-1) == INVALID and fwd(f=f, ci=0) == INVALID
        assert fwd(f=f, co=0) == INVALID and fwd(f=f, s=0) == INVALID and fwd(f=f, s=1025) == INVALID
        assert fwd(f=f, dt=-1) == INVALID
        # an operand without a row list has a row for every position
        assert fwd(f=f, n=3) == INVALID
        assert fwd(f=f, m=2 ** 31, n=2 ** 31) == UNSUPPORTED
        assert fwd(f=f, m=0, n=0, x=None) == 0
    assert fwd(xr=P(258)) == INVALID

    def wgrad(x=P(256), dy=P(256), nx=4, ny=4, m=4, dw=P(256), xr=None):
        return L.spc_grouped_wgrad(x, dy, P(256), xr, None, 2, nx, ny, m, 8, 8, 0, dw, None, P(256), 1 << 40, None)

    assert wgrad(x=None) == INVALID and wgrad(dy=None) == INVALID and wgrad(dw=None) == INVALID
    assert wgrad(nx=3) == INVALID and wgrad(ny=3) == INVALID and wgrad(dw=P(260)) == INVALID
    assert wgrad(m=-1) == INVALID


def test_binding_refusals():
    x = torch.zeros(4, 8)
    seg = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.spc_row_segments(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        binding.spc_row_segments(torch.zeros(4, 1, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        binding.spc_group_norm_fwd(x, None, None, seg, 2)
    with pytest.raises(ValueError):
        binding.spc_dropout_fwd(x, 0.5, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        binding.spc_grouped_fwd(x, torch.zeros(2, 8, 8), seg)
