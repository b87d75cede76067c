"""A transformer block's layers on the CPU: what their sources may hold, the steps of the rotary
positions, and the calls that are refused before anything is enqueued."""

import ctypes
import glob
import math
import os

import pytest
import torch

import sparse_convolution_hash_gb300 as spc
from sparse_convolution_hash_gb300 import binding
from sparse_convolution_hash_gb300 import build as libbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 6, 8
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return binding.lib()


def kernels():
    for f in sorted(glob.glob(os.path.join(libbuild.CSRC_BLOCK, "*.cu*"))):
        with open(f, encoding="utf-8") as fh:
            text = fh.read()
        for body in text.split("__global__")[1:]:
            yield f, body


def test_loads_fill_their_own_block_only_and_every_wait_has_a_limit():
    for f in glob.glob(os.path.join(libbuild.CSRC_BLOCK, "*")):
        with open(f, encoding="utf-8") as fh:
            text = fh.read()
        for piece in text.split("cp.async.bulk")[1:]:
            assert "multi" + "cast" not in piece.split('"')[0], f
        assert "mbarrier.try_wait" not in text and "mbarrier.test_wait" not in text, f  # only through the bounded one


def test_kernels_wait_for_the_one_before_them_first():
    """Kernels are set up beside the one before: none reads, writes or takes tensor memory before its end."""
    count = tensor = 0
    for f, body in kernels():
        count += 1
        at = body.find("wait_for_kernel_before();")
        assert at > 0, f
        assert "fetch(" not in body[:at] and "attn_tile(" not in body[:at], f
        if "tmem_alloc" in body:
            tensor += 1
            assert at < body.find("tmem_alloc"), f
    assert count >= 15 and tensor == 2


@pytest.mark.parametrize("pairs,base", [((10, 11, 11), 10000.0), ((1, 0, 3), 100.0), ((0, 0, 0), 2.0), ((128, 0, 0), 1.0)])
def test_rope_steps(L, pairs, base):
    steps = spc.spc_rope_steps(pairs, base)
    want = [base ** (-j / p) / (2 * math.pi) for p in pairs for j in range(p)]
    assert steps.dtype is torch.int64 and len(steps) == len(want)
    # the steps are whole; float64's own power has an exponent j / p off by 2^-53, so it is off by ln(base) times that,
    # and the power, 2 pi and the quotient add a rounding each
    for got, w in zip(steps.tolist(), want):
        assert abs(got / 2.0 ** 64 - w) <= 2.0 ** -53 * (4 + math.log(base)) * w + 2.0 ** -65


def test_rope_steps_refusals(L):
    for pairs, base in (((1, 2, 3), 0.5), ((1, 2, 3), math.nan), ((1, 2, 3), math.inf), ((100, 20, 9), 10.0)):
        with pytest.raises(spc.SpcError):
            spc.spc_rope_steps(pairs, base)
    for pairs in ((1, 2), (1, -2, 3)):
        with pytest.raises(ValueError):
            spc.spc_rope_steps(pairs)


def p(v):
    return None if v is None else ctypes.c_void_p(v)


def test_layer_norm_refusals(L):
    def fwd(x=256, ga=256, be=256, n=4, c=8, eps=1e-5, dt=F32, y=512, mean=1024, rstd=2048):
        return L.spc_layer_norm_fwd(p(x), p(ga), p(be), n, c, eps, dt, p(y), p(mean), p(rstd), None)

    for bad in (dict(x=None), dict(x=258), dict(x=257, dt=F16), dict(y=None), dict(mean=None), dict(rstd=1026), dict(ga=258), dict(be=257),
                dict(n=-1), dict(c=0), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(dt=3)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(n=1 << 60, c=16) == UNSUPPORTED
    assert fwd(n=0, x=None, y=None, mean=None, rstd=None) == OK
    need = L.spc_layer_norm_workspace_size(100, 64)
    assert need > 0 and L.spc_layer_norm_workspace_size(-1, 4) == 0 and L.spc_layer_norm_workspace_size(1, 0) == 0

    def bwd(dy=256, x=256, n=100, c=64, dx=512, dg=1024, db=2048, ws=4096, size=need, mean=256):
        return L.spc_layer_norm_bwd(p(dy), p(x), None, p(mean), p(256), n, c, F32, p(dx), p(dg), p(db), p(ws), size, None)

    for bad in (dict(dy=None), dict(dy=258), dict(x=None), dict(dx=None), dict(dg=1026), dict(db=2049), dict(mean=None)):
        assert bwd(**bad) == INVALID, bad
    for bad in (dict(ws=None), dict(ws=4100), dict(size=need - 1)):
        assert bwd(**bad) == WORKSPACE, bad


def test_rope_refusals(L):
    steps = (ctypes.c_uint64 * 8)()

    def call(f=L.spc_rope_fwd, x=256, ldx=16, coords=256, pairs=(2, 2, 2), st=steps, n=4, heads=1, d=16, dt=F32, y=512, ldy=16):
        return f(p(x), ldx, p(coords), (ctypes.c_int32 * 3)(*pairs), st and ctypes.addressof(st), n, heads, d, dt, p(y), ldy, None)

    for f in (L.spc_rope_fwd, L.spc_rope_bwd):
        for bad in (dict(x=None), dict(x=258), dict(y=None), dict(coords=None), dict(coords=264), dict(ldx=15), dict(ldy=8), dict(n=-1),
                    dict(heads=-1), dict(d=0), dict(dt=7), dict(pairs=(-1, 2, 2)), dict(pairs=(3, 3, 3)), dict(st=None),
                    dict(y=256, ldy=24), dict(ldx=BIG * BIG // 4)):
            assert call(f, **bad) == INVALID, bad
        assert call(f, d=400, ldx=400, ldy=400, pairs=(100, 50, 50)) == UNSUPPORTED
        for big in (dict(heads=2 ** 31 - 1, d=1, pairs=(0, 0, 0)), dict(d=2 ** 31 - 1)):
            assert call(f, n=1, ldx=2 ** 31, ldy=2 ** 31, **big) == UNSUPPORTED
        assert call(f, n=0, x=None, y=None, coords=None) == OK and call(f, heads=0, ldx=0, ldy=0) == OK


def test_route_refusals(L):
    def fwd(logits=256, bias=None, n=4, e=16, k=2, score=0, groups=1, kept=1, scale=1.0, dt=F32, expert=512, gate=1024):
        return L.spc_route_fwd(p(logits), p(bias), n, e, k, score, groups, kept, 1, scale, dt, p(expert), p(gate), None)

    for bad in (dict(logits=None), dict(logits=258), dict(bias=258), dict(n=-1), dict(e=0), dict(k=0), dict(k=17), dict(score=2),
                dict(groups=0), dict(groups=5), dict(groups=4, kept=0), dict(groups=4, kept=5), dict(groups=8, kept=1, k=3),
                dict(scale=math.inf), dict(scale=math.nan), dict(dt=5), dict(expert=None), dict(expert=514), dict(gate=None), dict(gate=1025)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(e=1025) == UNSUPPORTED and fwd(e=64, k=33) == UNSUPPORTED
    assert fwd(n=0, logits=None, expert=None, gate=None) == OK

    def bwd(dgate=256, logits=256, expert=256, n=4, e=16, k=2, score=1, scale=1.0, dt=F32, dl=512):
        return L.spc_route_bwd(p(dgate), p(logits), p(expert), n, e, k, score, 1, scale, dt, p(dl), None, None)

    for bad in (dict(dgate=None), dict(logits=None), dict(expert=None), dict(expert=257), dict(dl=None), dict(dl=256), dict(k=0),
                dict(score=-1), dict(scale=math.nan), dict(dt=9)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=0, dgate=None, logits=None, expert=None, dl=None) == OK


def test_attention_refusals(L):
    def args(q=256, ldq=64, k=256, ldk=64, v=256, ldv=64, sq=256, sk=256, S=2, nq=10, nk=10, hq=2, hk=2, d=32, scale=0.5, dt=BF16):
        return [p(q), ldq, p(k), ldk, p(v), ldv], [p(sq), p(sk), S, nq, nk, hq, hk, d, scale, dt]

    def fwd(o=1024, ldo=64, lse=2048, ws=4096, size=BIG, **kw):
        a, b = args(**kw)
        return L.spc_attention_fwd(*a, *b, p(o), ldo, p(lse), None, p(ws), size, None)

    def bwd(do=8192, lddo=64, o=1024, ldo=64, lse=2048, dq=16384, lddq=64, dk=32768, lddk=64, dv=65536, lddv=64, ws=4096, size=BIG, **kw):
        a, b = args(**kw)
        return L.spc_attention_bwd(p(do), lddo, *a, p(o), ldo, p(lse), *b, p(dq), lddq, p(dk), lddk, p(dv), lddv, None, p(ws), size, None)

    common = (dict(q=None), dict(q=257), dict(k=None), dict(v=None), dict(ldq=63), dict(ldk=40), dict(ldv=0), dict(sq=None), dict(sk=None),
              dict(sq=258), dict(S=0), dict(nq=-1), dict(nk=-1), dict(hq=0), dict(hk=0), dict(hq=3), dict(d=0), dict(scale=0.0),
              dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(dt=4), dict(o=None), dict(ldo=1), dict(lse=None), dict(lse=2050))
    for bad in common + (dict(o=256),):
        assert fwd(**bad) == INVALID, bad
    for bad in common + (dict(do=None), dict(lddo=3), dict(dq=None), dict(dk=None), dict(dv=32771), dict(lddq=4), dict(lddk=4), dict(lddv=4),
                         dict(dq=256), dict(dk=1024), dict(dv=16384), dict(dk=8192)):
        assert bwd(**bad) == INVALID, bad
    for f in (fwd, bwd):
        assert f(d=129, ldq=258, ldk=258, ldv=258, ldo=258, **({} if f is fwd else dict(lddo=258, lddq=258, lddk=258, lddv=258))) == UNSUPPORTED
        for n in (1 << 31, (1 << 31) - 128):
            assert f(nq=n) == UNSUPPORTED and f(nk=n) == UNSUPPORTED
    # few queries over many keys are split: a workspace
    few = dict(nq=2, nk=100000, S=1)
    need = L.spc_attention_workspace_size(2, 100000, 1, 2, 2, 32, BF16, 0)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=4097), dict(size=need - 1)):
        assert fwd(**few, **bad) == WORKSPACE, bad
    for bad in (dict(ws=None), dict(size=0)):
        assert bwd(**bad) == WORKSPACE
    size = L.spc_attention_workspace_size
    assert size(100000, 100000, 1, 8, 8, 64, BF16, 0) == 0  # many queries: none
    assert size(-1, 1, 1, 1, 1, 1, 0, 0) == 0 and size(1, 1, 1, 3, 2, 1, 0, 0) == 0 and size(1, 1, 1, 1, 1, 129, 0, 1) == 0
    assert size(1 << 40, 1, 1, 1, 1, 8, 0, 1) == 0 and size(1, (1 << 31) - 128, 1, 1, 1, 8, 0, 1) == 0


def test_tensors_on_the_host_are_refused(L):
    x = torch.zeros(4, 8)
    h = torch.zeros(4, 2, 8)
    seg = torch.tensor([0, 4], dtype=torch.int32)
    calls = [lambda: spc.spc_layer_norm_fwd(x, None, None), lambda: spc.spc_layer_norm_bwd(x, x, None, x[:, 0], x[:, 0]),
             lambda: spc.spc_rope_fwd(h, torch.zeros(4, 4, dtype=torch.int32), spc.spc_rope_steps((1, 1, 1)), (1, 1, 1)),
             lambda: spc.spc_route_fwd(x, 2), lambda: spc.spc_route_bwd(x[:, :2], x, x[:, :2]),
             lambda: spc.spc_attention_fwd(h, h, h, seg), lambda: spc.spc_attention_bwd(h, h, h, h, h, x[:, :2], seg)]
    for f in calls:
        with pytest.raises(ValueError):
            f()
