"""The plain float64 forms of a transformer block's layers against autograd and differences (CPU)."""

import math

import pytest
import torch

import block_ref as ref


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def test_layer_norm_is_torchs_and_its_gradient_autograds():
    g = gen(1)
    x, ga, be, dy = normal(g, 7, 13).float(), normal(g, 13).float(), normal(g, 13).float(), normal(g, 7, 13).float()
    (y, mean, rstd), _ = ref.layer_norm_fwd(x, ga, be, 1e-5)
    z = [t.double().requires_grad_() for t in (x, ga, be)]
    want = torch.nn.functional.layer_norm(z[0], (13,), z[1], z[2], 1e-5)
    assert torch.allclose(y, want, atol=1e-12)
    got = ref.layer_norm_bwd(dy, x, ga, mean, rstd)[0]
    for a, b in zip(got, torch.autograd.grad((want * dy.double()).sum(), z)):
        assert torch.allclose(a, b, atol=1e-10)


def test_rope_turns_by_distance_only_and_back():
    g = gen(2)
    pairs, n = (2, 3, 1), 5
    x = normal(g, n, 2, 14).float()
    coords = torch.randint(-50, 50, (n, 4), generator=g, dtype=torch.int32)
    y, _ = ref.rope(x, coords, pairs, 100.0)
    assert torch.allclose(y.norm(dim=2), x.double().norm(dim=2))
    assert torch.equal(y[:, :, 12:], x.double()[:, :, 12:])
    # products of turned rows hang on the difference of their cells
    q, k = x[:1].expand(2, 2, 14), x[1:2].expand(2, 2, 14)
    c = torch.tensor([[0, 3, 4, 5], [0, 10, 24, -5]], dtype=torch.int32)
    far = c + torch.tensor([0, 7, -9, 2], dtype=torch.int32)
    a = (ref.rope(q, c, pairs, 100.0)[0] * ref.rope(k, far, pairs, 100.0)[0]).sum(2)
    assert torch.allclose(a[0], a[1])
    back, _ = ref.rope(y.float(), coords, pairs, 100.0, back=True)
    assert torch.allclose(back, x.double(), atol=1e-5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_autograds(score, renorm):
    g = gen(3)
    logits, dgate = normal(g, 6, 8).float(), normal(g, 6, 3).float()
    (expert, gate), _ = ref.route_fwd(logits, 3, score, None, 1, 1, renorm, 1.7)
    z = logits.double().requires_grad_()
    p = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    w = p.gather(1, expert.long())
    w = 1.7 * (w / w.sum(1, keepdim=True) if renorm else w)
    assert torch.allclose(gate, w)
    assert torch.equal(expert.long(), logits.topk(3, 1).indices)
    want = torch.autograd.grad((w * dgate.double()).sum(), z)[0]
    assert torch.allclose(ref.route_bwd(dgate, logits, expert, score, renorm, 1.7)[0], want, atol=1e-12)


def test_route_ties_groups_and_missing_experts():
    x = torch.tensor([[1.0, 1.0, 0.5, 1.0], [-math.inf, math.nan, 2.0, -math.inf], [-math.inf] * 4])
    (expert, gate), _ = ref.route_fwd(x, 2, "softmax", None, 1, 1, True, 1.0)
    assert expert.tolist() == [[0, 1], [2, -1], [-1, -1]]
    assert gate.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]]
    # the second group has the better pair, the first the best expert
    x = torch.tensor([[3.0, -9.0, 2.0, 2.0]])
    (expert, _), _ = ref.route_fwd(x, 2, "sigmoid", None, 2, 1, True, 1.0)
    assert expert.tolist() == [[2, 3]]
    (expert, _), _ = ref.route_fwd(x, 1, "sigmoid", torch.tensor([0.0, 5.0, 0.0, 0.0]), 1, 1, True, 1.0)
    assert expert.tolist() == [[1]]


def test_attention_is_the_formulas_and_its_gradient_autograds():
    g = gen(4)
    q, k, v = (normal(g, n, h, 5).float() for n, h in ((9, 4), (11, 2), (11, 2)))
    dout = normal(g, 9, 4, 5).float()
    seg, seg_k = [0, 3, 3, 7, 9], [1, 5, 6, 6, 11]  # a segment without queries, one without keys
    z = [t.double().requires_grad_() for t in (q, k, v)]
    want = torch.zeros(9, 4, 5, dtype=torch.float64)
    for s in range(4):
        a, b = slice(seg[s], seg[s + 1]), slice(seg_k[s], seg_k[s + 1])
        if b.stop > b.start:
            kk, vv = (t[b].repeat_interleave(2, 1) for t in z[1:])
            p = torch.softmax(torch.einsum("qhd,khd->hqk", z[0][a], kk) * 0.3, 2)
            want = torch.cat([want[:a.start], torch.einsum("hqk,khd->qhd", p, vv), want[a.stop:]])
    (o, lse), _ = ref.attention_fwd(q, k, v, seg, seg_k, 0.3, False)
    assert torch.allclose(o, want) and bool((lse[3:7] == -math.inf).all()) and bool((o[3:7] == 0).all())
    got = ref.attention_bwd(dout, q, k, v, o, lse, seg, seg_k, 0.3, False)[0]
    for a, b in zip(got, torch.autograd.grad((want * dout.double()).sum(), z)):
        assert torch.allclose(a, b, atol=1e-12)
