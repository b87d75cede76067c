"""The example block (norm, conv, norm, routed experts, dropout, residual) against the same block
written with torch autograd in float64 on the CPU: output and every gradient.

Bounds are normwise.  fp32: about ten steps, each summing at most 27 x 64 products, so
10 x 27 x 64 x 2^-24 < 2e-3 at worst and a fiftieth of that for rounding errors of either
sign: 4e-5.  bf16: about ten roundings of 2^-8 on the way to the output and twenty to the
gradients, of either sign: sqrt(20) 2^-8 with a factor of two, 3.5e-2.  What the
device decided where a decision jumps, a voxel's expert and the sign that a relu
saw, is given to the reference: a rounding that turns one moves a gradient by its
whole size."""

import os
import sys

import numpy as np
import pytest
import torch

import layers_ref as ref
import oracle
import sparse_convolution_hash_gb300 as spc
from gpu_util import DT, dev, rand_coords

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def reference(block, x, coords, batch, grid, expert, positive, mask, dy):
    """y and gradients of the block by autograd, float64."""
    names = ("gamma1", "beta1", "gamma2", "beta2", "conv", "router", "w1", "w2")
    p = {k: getattr(block, k).detach().cpu().double().requires_grad_() for k in names}
    x = x.detach().cpu().double().requires_grad_()
    imap, _ = oracle.subm_map(coords, batch, grid)
    sample = torch.from_numpy(coords[:, 0].astype(np.int64))

    def norm(h, gamma, beta):
        out = torch.zeros_like(h)
        for s in range(batch):
            at = torch.nonzero(sample == s)[:, 0]
            z = torch.nn.functional.group_norm(h[at].T[None], block.groups, gamma, beta, 1e-5)[0].T
            out = out.index_put((at,), torch.nn.functional.silu(z))
        return out

    h1 = norm(x, p["gamma1"], p["beta1"])
    h2 = torch.zeros(x.shape[0], p["conv"].shape[2], dtype=torch.float64)
    for k in range(27):
        hit = torch.from_numpy(np.nonzero(imap[k] >= 0)[0])
        h2 = h2.index_add(0, hit, h1[torch.from_numpy(imap[k][imap[k] >= 0].astype(np.int64))] @ p["conv"][k])
    h3 = norm(h2, p["gamma2"], p["beta2"])
    prob = torch.softmax(h3 @ p["router"], 1)
    gate = prob.gather(1, expert[:, None])
    v = torch.zeros_like(h3)
    for e in range(p["w1"].shape[0]):
        at = torch.nonzero(expert == e)[:, 0]
        v = v.index_put((at,), (h3[at] @ p["w1"][e] * positive[at]) @ p["w2"][e])
    y = x + torch.where(mask, gate * v / (1 - block.p), torch.zeros_like(v))
    y.backward(dy.cpu().double())
    return y.detach(), x.grad, {k: t.grad for k, t in p.items()}


@pytest.mark.parametrize("dtype,tol", [("f32", 4e-5), ("bf16", 3.5e-2)])
def test_expert_block_matches_autograd(dtype, tol):
    from expert_block import ExpertBlock, Scene

    g = np.random.default_rng(5)
    n, c, batch, grid = 700, 64, 3, (10, 9, 11)
    coords = rand_coords(g, n, batch, grid)  # rows in no order
    block = ExpertBlock(c, 128, 5, 8, 0.25, DT[dtype], dev())
    with torch.no_grad():
        for name in ("gamma1", "beta1", "gamma2", "beta2"):
            getattr(block, name).add_(torch.from_numpy(g.standard_normal(c) * 0.2).float().to(dev()))
    x = torch.from_numpy(g.standard_normal((n, c))).to(DT[dtype]).to(dev())
    dy = torch.from_numpy(g.standard_normal((n, c))).to(DT[dtype]).to(dev())
    rng = torch.tensor([11, 22], device=dev())
    scene = Scene(torch.from_numpy(coords).to(dev()), batch, grid)
    y, saved = block.forward(x, scene, rng)
    dx, grads = block.backward(dy, scene, saved)
    torch.cuda.synchronize()
    mask = torch.from_numpy(ref.dropout_words(11, 22, 0, n * c) >= np.uint64(2 ** 30)).view(n, c)
    want = reference(block, x, coords, batch, grid, saved[10].cpu(), (saved[13] > 0).cpu().double(), mask, dy)

    def off(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())

    assert off(y, want[0]) < tol
    assert off(dx, want[1]) < tol
    for name, grad in grads.items():
        assert off(grad, want[2][name]) < tol, name
