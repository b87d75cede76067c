"""A transformer block over the voxels of a batch with routed experts, forward and backward.

    h  = layer_norm(x),  (q, k, v) = h Wqkv
    q, k turned by the voxels' (z, y, x) cells
    x1 = x + attention(q, k, v) Wo          each voxel to the voxels of its own sample
    h2 = layer_norm(x1)
    e, g = the top k experts of each voxel and their weights, from h2 R
    y  = x1 + sum over k of g relu(h2 W1[e]) W2[e]

The dense products, relu and the sums are torch; every other step is a call of the library, and the
backward pass is written out with the matching gradients.  Rows of a sample lie together (coordinates sorted
by their batch index).

    python examples/voxel_transformer.py      one training step on the strided voxels of four shells, bf16, timed
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_convolution_hash_gb300 as spc  # noqa: E402


class VoxelTransformerBlock:
    def __init__(self, channels: int, heads: int, kv_heads: int, hidden: int, experts: int, top_k: int, dtype, device, seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device=device, dtype=dtype)

        self.heads, self.kv_heads, self.d, self.top_k = heads, kv_heads, channels // heads, top_k
        third = self.d // 6
        self.pairs = (self.d // 2 - 2 * third, third, third)
        self.steps = spc.spc_rope_steps(self.pairs)
        self.gamma1 = torch.ones(channels, device=device)
        self.beta1 = torch.zeros(channels, device=device)
        self.gamma2 = torch.ones(channels, device=device)
        self.beta2 = torch.zeros(channels, device=device)
        self.qkv = normal(channels, (heads + 2 * kv_heads) * self.d, std=channels ** -0.5)
        self.out = normal(channels, channels, std=channels ** -0.5)
        self.router = normal(channels, experts, std=channels ** -0.5)
        self.w1 = normal(experts, channels, hidden, std=channels ** -0.5)
        self.w2 = normal(experts, hidden, channels, std=hidden ** -0.5)

    def _parts(self, qkv):
        a, b = self.heads, self.heads + self.kv_heads
        return qkv[:, :a], qkv[:, a:b], qkv[:, b:]

    def forward(self, x: torch.Tensor, coords: torch.Tensor, seg: torch.Tensor):
        """y, and what the backward pass needs.  seg: the offsets of the samples' rows."""
        n, c = x.shape
        h, mean1, rstd1 = spc.spc_layer_norm_fwd(x, self.gamma1, self.beta1)
        qkv = (h @ self.qkv).view(n, -1, self.d)
        turned = qkv[:, :self.heads + self.kv_heads]
        spc.spc_rope_fwd(turned, coords, self.steps, self.pairs, out=turned)
        o, lse = spc.spc_attention_fwd(*self._parts(qkv), seg)
        x1 = x + o.view(n, c) @ self.out
        h2, mean2, rstd2 = spc.spc_layer_norm_fwd(x1, self.gamma2, self.beta2)
        logits = h2 @ self.router
        expert, gate = spc.spc_route_fwd(logits, self.top_k)
        to, order = spc.spc_row_segments(expert.view(-1), self.router.shape[1])
        rows = order // self.top_k  # a slot's voxel
        a = torch.relu(spc.spc_grouped_fwd(h2, self.w1, to, x_rows=rows, y_rows=order))
        v = spc.spc_grouped_fwd(a, self.w2, to, x_rows=order, y_rows=order).view(n, self.top_k, c)
        y = x1 + (v.float() * gate[:, :, None]).sum(1).to(x.dtype)
        return y, (x, h, mean1, rstd1, qkv, o, lse, x1, h2, mean2, rstd2, logits, expert, gate, to, order, rows, a, v)

    def backward(self, dy: torch.Tensor, coords: torch.Tensor, seg: torch.Tensor, saved):
        """dx and the gradients of the parameters, by name."""
        x, h, mean1, rstd1, qkv, o, lse, x1, h2, mean2, rstd2, logits, expert, gate, to, order, rows, a, v = saved
        n, c = x.shape
        grads = {}
        dgate = (v.float() * dy.float()[:, None]).sum(2)
        dv = (gate[:, :, None] * dy.float()[:, None]).to(dy.dtype).view(-1, c)
        slots = dict(x_rows=order, y_rows=order)
        grads["w2"] = spc.spc_grouped_wgrad(a, dv, to, **slots)
        du = spc.spc_grouped_dgrad(dv, self.w2, to, **slots) * (a > 0)
        grads["w1"] = spc.spc_grouped_wgrad(h2, du, to, x_rows=rows, y_rows=order)
        dh2 = spc.spc_grouped_dgrad(du, self.w1, to, **slots).view(n, self.top_k, c).sum(1)
        dlogits = spc.spc_route_bwd(dgate, logits, expert)
        grads["router"] = h2.T @ dlogits
        dx1, grads["gamma2"], grads["beta2"] = spc.spc_layer_norm_bwd(dh2 + dlogits @ self.router.T, x1, self.gamma2, mean2, rstd2)
        dx1 = dx1 + dy
        grads["out"] = o.view(n, c).T @ dx1
        do = (dx1 @ self.out.T).view_as(o)
        dqkv = torch.empty_like(qkv)
        dq, dk, dvv = self._parts(dqkv)
        spc.spc_attention_bwd(do, *self._parts(qkv), o, lse, seg, dq=dq, dk=dk, dv=dvv)
        turned = dqkv[:, :self.heads + self.kv_heads]
        spc.spc_rope_bwd(turned, coords, self.steps, self.pairs, out=turned)
        flat = dqkv.view(n, -1)
        grads["qkv"] = h.T @ flat
        dx, grads["gamma1"], grads["beta1"] = spc.spc_layer_norm_bwd(flat @ self.qkv.T, x, self.gamma1, mean1, rstd1)
        return dx + dx1, grads


def main():
    import scenes

    dev = torch.device("cuda:0")
    w = scenes.workload("shell192x4_train_bf16")
    # two strided steps down, where samples are short enough to attend to themselves
    coords, grid = torch.from_numpy(w["coords"]).to(dev), w["shape"]
    for _ in range(2):
        coords, grid = spc.spc_strided_out_coords(coords, w["batch"], grid, 3, 2, 1, 1)[0], spc.spc_out_shape(grid)
    seg, _ = spc.spc_row_segments(coords[:, 0], w["batch"], with_order=False)
    block = VoxelTransformerBlock(channels=512, heads=8, kv_heads=8, hidden=1024, experts=8, top_k=2, dtype=torch.bfloat16, device=dev)
    torch.manual_seed(0)
    x, dy = (torch.randn(coords.shape[0], 512, device=dev).to(torch.bfloat16) for _ in range(2))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(6):
        start.record()
        y, saved = block.forward(x, coords, seg)
        dx, grads = block.backward(dy, coords, seg, saved)
        end.record()
        torch.cuda.synchronize()
        print(f"step {step}: {start.elapsed_time(end):.2f} ms, rows of each sample {seg.diff().tolist()}, |y| {float(y.float().norm()):.1f}, "
              f"|dx| {float(dx.float().norm()):.1f}")


if __name__ == "__main__":
    main()
