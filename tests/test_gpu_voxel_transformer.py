"""The example transformer block against the same block written with torch autograd in float64 on the
CPU: output and every gradient.

Bounds are normwise.  fp32: some fifteen steps, each summing at most 128 products (attention: 300 keys), with
rounding errors of either sign a fiftieth of 15 x 300 x 2^-24 < 3e-4: 1e-5, doubled for the gradients that follow.  bf16: about
fifteen roundings of 2^-8 to the output and thirty to the gradients, of either sign: sqrt(30) 2^-8 with a factor
of two, 4.3e-2.  What the device decided where a decision jumps, a voxel's experts and the sign that a relu saw, is
given to the reference."""

import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import DT, dev, rand_coords

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def reference(block, x, coords, seg, expert, positive, dy):
    names = ("gamma1", "beta1", "gamma2", "beta2", "qkv", "out", "router", "w1", "w2")
    p = {k: getattr(block, k).detach().cpu().double().requires_grad_() for k in names}
    x = x.detach().cpu().double().requires_grad_()
    n, c = x.shape
    d, heads, kv, top = block.d, block.heads, block.kv_heads, block.top_k
    h = torch.nn.functional.layer_norm(x, (c,), p["gamma1"], p["beta1"], 1e-5)
    qkv = (h @ p["qkv"]).view(n, -1, d)
    axis = torch.tensor([1 + a for a in range(3) for _ in range(block.pairs[a])])
    freq = torch.tensor([10000.0 ** (-j / q) for q in block.pairs for j in range(q)], dtype=torch.float64)
    angle = torch.from_numpy(coords).double()[:, axis] * freq
    pairs = len(freq)

    def turn(t):
        z = torch.view_as_complex(t[:, :, :2 * pairs].reshape(n, -1, pairs, 2)) * torch.polar(torch.ones_like(angle), angle)[:, None]
        return torch.cat([torch.view_as_real(z).reshape(n, -1, 2 * pairs), t[:, :, 2 * pairs:]], 2)

    q, k, v = turn(qkv[:, :heads]), turn(qkv[:, heads:heads + kv]), qkv[:, heads + kv:]
    k, v = (t.repeat_interleave(heads // kv, 1) for t in (k, v))
    o = []
    for a, b in zip(seg[:-1], seg[1:]):
        s = torch.softmax(torch.einsum("qhd,khd->hqk", q[a:b], k[a:b]) * d ** -0.5, 2)
        o.append(torch.einsum("hqk,khd->qhd", s, v[a:b]))
    x1 = x + torch.cat(o).reshape(n, c) @ p["out"]
    h2 = torch.nn.functional.layer_norm(x1, (c,), p["gamma2"], p["beta2"], 1e-5)
    prob = torch.softmax(h2 @ p["router"], 1).gather(1, expert)
    gate = prob / prob.sum(1, keepdim=True)
    slot = h2.repeat_interleave(top, 0)
    out = torch.zeros_like(slot)
    flat = expert.reshape(-1)
    for e in range(p["w1"].shape[0]):
        at = torch.nonzero(flat == e)[:, 0]
        out = out.index_put((at,), (slot[at] @ p["w1"][e] * positive[at]) @ p["w2"][e])
    y = x1 + (out.view(n, top, c) * gate[:, :, None]).sum(1)
    y.backward(dy.cpu().double())
    return y.detach(), x.grad, {k: t.grad for k, t in p.items()}


@pytest.mark.parametrize("dtype,tol", [("f32", 2e-5), ("bf16", 4.3e-2)])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (4, 1)])
def test_voxel_transformer_matches_autograd(heads, kv_heads, dtype, tol):
    import sparse_convolution_hash_gb300 as spc
    from voxel_transformer import VoxelTransformerBlock

    g = np.random.default_rng(6)
    n, c, batch = 700, 128, 3
    coords = rand_coords(g, n, batch, (10, 30, 20))
    coords = np.ascontiguousarray(coords[np.argsort(coords[:, 0], kind="stable")])
    block = VoxelTransformerBlock(c, heads, kv_heads, 96, 5, 2, DT[dtype], dev())
    for name in ("gamma1", "beta1", "gamma2", "beta2"):
        getattr(block, name).add_(torch.from_numpy(g.standard_normal(c) * 0.2).float().to(dev()))
    x, dy = (torch.from_numpy(g.standard_normal((n, c))).to(DT[dtype]).to(dev()) for _ in range(2))
    t = torch.from_numpy(coords).to(dev())
    seg, _ = spc.spc_row_segments(t[:, 0], batch, with_order=False)
    y, saved = block.forward(x, t, seg)
    dx, grads = block.backward(dy, t, seg, saved)
    torch.cuda.synchronize()
    want = reference(block, x, coords, seg.tolist(), saved[12].cpu().long(), (saved[17] > 0).cpu().double(), dy)

    def off(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())

    assert off(y, want[0]) < tol
    assert off(dx, want[1]) < tol
    assert set(grads) == set(want[2])
    for name, grad in grads.items():
        assert off(grad, want[2][name]) < tol, name
