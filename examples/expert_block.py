"""A residual block of a sparse network with routed experts, forward and backward.

    h1 = silu(group_norm(x))             per sample
    h2 = submanifold conv 3x3x3 (h1)
    h3 = silu(group_norm(h2))
    e  = the voxel's expert, the largest of softmax(h3 R); its probability is the gate
    v  = relu(h3 W1[e]) W2[e]            products grouped by expert
    y  = x + dropout(gate v)

Every step but the router's small dense product and the elementwise relu and gate is a call of
the library; the backward pass is written out with the matching gradients.

    python examples/expert_block.py      one training step on the 4 x 192^3 shells, bf16, timed
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_convolution_hash_gb300 as spc  # noqa: E402


class Scene:
    """What a batch of coordinates gives once: the conv's indice map and the rows of each sample."""

    def __init__(self, coords: torch.Tensor, batch: int, grid):
        self.map = spc.spc_build_indice_map(coords, batch, grid)
        spc.check_status(self.map["status"], "indice map")
        # rows may lie in any order: the samples' rows are grouped through a list
        self.seg, self.order = spc.spc_row_segments(coords[:, 0], batch)


class ExpertBlock:
    def __init__(self, channels: int, hidden: int, experts: int, groups: int, p: float, dtype, device, seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device=device, dtype=dtype)

        self.groups, self.p = groups, p
        self.gamma1 = torch.ones(channels, device=device)
        self.beta1 = torch.zeros(channels, device=device)
        self.gamma2 = torch.ones(channels, device=device)
        self.beta2 = torch.zeros(channels, device=device)
        self.conv = normal(27, channels, channels, std=(27 * channels) ** -0.5)
        self.router = normal(channels, experts, std=channels ** -0.5)
        self.w1 = normal(experts, channels, hidden, std=channels ** -0.5)
        self.w2 = normal(experts, hidden, channels, std=hidden ** -0.5)

    def forward(self, x: torch.Tensor, scene: Scene, rng: torch.Tensor):
        """y, and what the backward pass needs.  rng: seed and offset of this step's dropout."""
        k = dict(act=spc.SPC_ACT_SILU, order=scene.order)
        h1, mean1, rstd1 = spc.spc_group_norm_fwd(x, self.gamma1, self.beta1, scene.seg, self.groups, **k)
        h2 = spc.spc_conv_fwd(h1, self.conv, None, scene.map["imap"], scene.map["mask"])
        h3, mean2, rstd2 = spc.spc_group_norm_fwd(h2, self.gamma2, self.beta2, scene.seg, self.groups, **k)
        prob = torch.softmax((h3 @ self.router).float(), 1)
        gate, expert = prob.max(1)
        seg, order = spc.spc_row_segments(expert.to(torch.int32), self.router.shape[1])
        rows = dict(x_rows=order, y_rows=order)
        u = spc.spc_grouped_fwd(h3, self.w1, seg, **rows)
        a = torch.relu(u)
        v = spc.spc_grouped_fwd(a, self.w2, seg, **rows)
        y = spc.spc_dropout_fwd(v * gate[:, None].to(v.dtype), self.p, rng, residual=x)
        return y, (x, h1, mean1, rstd1, h2, h3, mean2, rstd2, prob, gate, expert, seg, order, a, v, rng)

    def backward(self, dy: torch.Tensor, scene: Scene, saved):
        """dx and the gradients of the parameters, by name."""
        x, h1, mean1, rstd1, h2, h3, mean2, rstd2, prob, gate, expert, seg, order, a, v, rng = saved
        k = dict(act=spc.SPC_ACT_SILU, order=scene.order)
        rows = dict(x_rows=order, y_rows=order)
        grads = {}
        dvg = spc.spc_dropout_bwd(dy, self.p, rng)
        dv = dvg * gate[:, None].to(dvg.dtype)
        dgate = (dvg.float() * v.float()).sum(1)
        grads["w2"] = spc.spc_grouped_wgrad(a, dv, seg, **rows)
        du = spc.spc_grouped_dgrad(dv, self.w2, seg, **rows) * (a > 0)
        grads["w1"] = spc.spc_grouped_wgrad(h3, du, seg, **rows)
        dh3 = spc.spc_grouped_dgrad(du, self.w1, seg, **rows)
        chosen = torch.zeros_like(prob).scatter_(1, expert[:, None], 1.0)
        dlogits = ((chosen - prob) * (gate * dgate)[:, None]).to(h3.dtype)
        grads["router"] = h3.T @ dlogits
        dh3 = dh3 + dlogits @ self.router.T
        dh2, grads["gamma2"], grads["beta2"] = spc.spc_group_norm_bwd(
            dh3, h2, self.gamma2, self.beta2, mean2, rstd2, scene.seg, self.groups, **k)
        imap = scene.map["imap"]
        grads["conv"] = spc.spc_conv_wgrad(h1, dh2, imap, 27)
        dh1 = spc.spc_conv_dgrad(dh2, self.conv, imap, spc.SPC_MAP_SUBM_MIRROR, x.shape[0], mask=scene.map["mask"])
        dx, grads["gamma1"], grads["beta1"] = spc.spc_group_norm_bwd(
            dh1, x, self.gamma1, self.beta1, mean1, rstd1, scene.seg, self.groups, **k)
        return dx + dy, grads


def main():
    import scenes

    dev = torch.device("cuda:0")
    w = scenes.workload("shell192x4_train_bf16")
    coords = torch.from_numpy(w["coords"]).to(dev)
    scene = Scene(coords, w["batch"], w["shape"])
    block = ExpertBlock(channels=64, hidden=256, experts=8, groups=16, p=0.1, dtype=torch.bfloat16, device=dev)
    torch.manual_seed(0)
    x, dy = w["x"].to(dev), torch.randn(coords.shape[0], 64, device=dev).to(torch.bfloat16)
    rng = torch.tensor([1234, 0], device=dev)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(6):
        rng = rng + torch.tensor([0, 1], device=dev)  # a new mask each step
        start.record()
        y, saved = block.forward(x, scene, rng)
        dx, grads = block.backward(dy, scene, saved)
        end.record()
        torch.cuda.synchronize()
        print(f"step {step}: {start.elapsed_time(end):.2f} ms, |y| {float(y.float().norm()):.1f}, "
              f"|dx| {float(dx.float().norm()):.1f}, rows of each expert {saved[11].diff().tolist()}")


if __name__ == "__main__":
    main()
