"""A transformer block's layers in the corners of their ranges.

Bounds are those of block_ref.py, or derived beside the test from the same arithmetic (E = 2^-24)."""

import math

import pytest
import torch

import sparse_convolution_hash_gb300 as spc
from gpu_util import dev
from test_gpu_block import TYPES, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def offsets(*seg):
    return torch.tensor(seg, dtype=torch.int32, device=dev())


# ------------------------------------------------------------------ no rows on one side
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hk", [(8, 8), (8, 2)])
@pytest.mark.parametrize("n", [1000, 20000])
def test_attention_gradients_where_one_side_has_no_rows(n, hq, hk, dtype):
    """Many rows on the other side, whose walk would be split."""
    q, k = (normal(gen(n), n, h, 16, dtype=dtype).to(dev()) for h in (hq, hk))
    none_q, none_k = q[:0], k[:0]
    no, all_ = offsets(0, 0), offsets(0, n)
    o, lse = spc.spc_attention_fwd(q, none_k, none_k, all_, seg_k=no)
    assert not o.any() and bool((lse == -math.inf).all())
    dq, dk, dv = spc.spc_attention_bwd(q, q, none_k, none_k, o, lse, all_, seg_k=no, dq=torch.full_like(q, 7))
    assert not dq.any() and dk.shape == dv.shape == none_k.shape
    o, lse = spc.spc_attention_fwd(none_q, k, k, no, seg_k=all_)
    dq, dk, dv = spc.spc_attention_bwd(none_q, none_q, k, k, o, lse, no, seg_k=all_, dk=torch.full_like(k, 7), dv=torch.full_like(k, 7))
    assert dq.shape == none_q.shape and not dk.any() and not dv.any()
