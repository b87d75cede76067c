"""The layers between convolutions, checked on the CPU: what their sources may hold, and
the arithmetic of their kernels that runs as plain host code."""

import ctypes
import glob
import os
import shutil
import subprocess

import numpy as np
import pytest

from sparse_convolution_hash_gb300 import binding
from sparse_convolution_hash_gb300 import build as libbuild


def test_no_load_fills_several_ctas():
    """The library runs on every GPU of a job: a bulk load goes to its own CTA only.  (A commit of the
    tensor core may arrive on both barriers of a CTA pair: it moves no data.)"""
    sources = [f for d in (libbuild.CSRC, libbuild.CSRC_LAYERS) for f in glob.glob(os.path.join(d, "*"))]
    assert sources
    for f in sources:
        with open(f, encoding="utf-8") as fh:
            text = fh.read()
        for piece in text.split("cp.async.bulk")[1:]:
            assert "multi" + "cast" not in piece.split('"')[0], f


def test_tensor_memory_is_taken_after_the_wait():
    """A kernel set up beside the one before it holds no tensor memory while it waits: the other may still
    have blocks to start that need some."""
    kernels = 0
    for f in glob.glob(os.path.join(libbuild.CSRC_LAYERS, "*.cu")):
        with open(f, encoding="utf-8") as fh:
            for body in fh.read().split("__global__")[1:]:
                if "tmem_alloc" in body:
                    kernels += 1
                    assert 0 <= body.find("wait_for_kernel_before();") < body.find("tmem_alloc"), f
    assert kernels == 2


# ------------------------------------------- the plan of the gradient by the weights
@pytest.fixture(scope="module")
def plan_check(tmp_path_factory):
    """tests/wgrad_plan_check.cpp, built with the host compiler: lines of cases to lines of findings."""
    cxx = shutil.which("g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(libbuild.nvcc())), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = str(tmp_path_factory.mktemp("plan") / "wgrad_plan_check")
    subprocess.run([cxx, "-std=c++20", "-O2", "-pthread", "-I", cuda, "-I", libbuild.INCLUDE, "-I", libbuild.CSRC,
                    "-I", libbuild.CSRC_LAYERS, os.path.join(os.path.dirname(__file__), "wgrad_plan_check.cpp"),
                    "-o", exe], check=True)

    def run(cases):
        text = "".join(f"{len(seg) - 1} {m} {tiles} {parts} {' '.join(map(str, seg))}\n" for m, tiles, parts, seg in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300, check=True).stdout
        return out.split("\n")[:-1]

    return run


def offsets(units):
    return [64 * sum(units[:i]) for i in range(len(units) + 1)]


# Tiles of a segment, CTAs, and 64-row units of each segment whose whole tiles fill the CTAs to levels that
# differ by orders of magnitude.
STEEP = [
    (94, 152, [1688, 57, 46711, 291, 2112, 2, 181, 489, 91, 449, 5, 1, 1053, 729, 6, 1296, 20691, 6238, 13, 1137,
      6, 134, 381, 391, 98835, 47, 1816, 2181, 52, 41006, 1, 1774, 268, 1, 19, 366, 130, 170, 4161, 21, 175542, 3,
      6525, 1555, 21, 29, 22, 4794, 26588, 2840, 428, 574, 2, 11, 2]),
    (105, 100, [113, 133690, 3, 17301, 12, 75, 2, 2518, 173, 23, 11346, 6, 1702, 136892, 4842930, 48720, 499, 10,
      6, 38, 249, 348, 1, 223, 497, 633, 3237, 253, 3, 16, 16, 146187, 3710, 601, 1194, 47, 256, 1, 140, 24, 52,
      54043, 3173, 6185, 415, 43930, 19307, 1631, 5, 63, 1732, 1260098, 16863, 32, 65136, 243, 109, 2, 3, 2, 1]),
]


@pytest.mark.parametrize("tiles,parts,units", STEEP)
def test_weight_gradient_plan_of_steep_segments(plan_check, tiles, parts, units):
    seg = offsets(units)
    assert [f.split(" ")[0] for f in plan_check([(seg[-1], tiles, parts, seg)])] == ["ok"]


def test_weight_gradient_plan_of_many_splits(plan_check):
    """Rows of every skew, with and without cut tiles, one CTA and more than there are tiles."""
    g = np.random.default_rng(0)
    cases = []
    for i in range(120):
        segments = int(g.integers(1, 200)) if i % 6 else 1024
        m, tiles = int(np.exp(g.uniform(0, 16))), int(np.exp(g.uniform(0, 4)))
        w = np.exp(g.uniform(0, 4) * g.standard_normal(segments))
        seg = np.concatenate([[0], np.cumsum(g.multinomial(m, w / w.sum()))]) + int(g.integers(0, 100))
        cases.append((m + 150, tiles, int(g.choice([1, 2, 16, 76, 152, 152, 192])), seg.tolist()))
    found = plan_check(cases)
    assert len(found) == len(cases)
    assert [f for f in found if not f.startswith("ok")] == []
    assert sum(f != "ok (0, 0)" for f in found) > 20  # tiles were cut


@pytest.mark.parametrize("segments,m,tiles", [(1024, 2 ** 31 - 2, 1), (1024, 300000000, 3), (200, 2 ** 31 - 2, 1),
                                              (1024, 2 ** 28 + 999, 2), (1024, 100000, 5)])
def test_weight_gradient_plan_of_offsets_out_of_order(plan_check, segments, m, tiles):
    """Offsets that go back and forth name every row hundreds of times: reported, and no piece or join
    leaves the tensors however many units that is."""
    seg = [0 if i % 2 == 0 else m for i in range(segments + 1)]
    assert plan_check([(m, tiles, 152, seg)])[0].startswith("ok") and plan_check([(m, tiles, 152, seg)])[0].endswith(", 10)")


# ----------------------------------------------------------------- refusals
def test_grouped_products_refuse_tensors_off_their_boundary():
    """16 bytes on tensor cores, four elements where rows are a multiple of four, else an element."""
    libbuild.build()
    L, P = binding.lib(), ctypes.c_void_p

    def codes(shift, c, dt):
        for at in range(3):
            p = [P(256), P(256), P(256)]
            p[at] = P(256 + shift)
            for f in (L.spc_grouped_fwd, L.spc_grouped_dgrad):
                yield f(p[0], p[1], P(256), None, None, 2, 4, 4, c, c, dt, p[2], None, None, 0, None)
            yield L.spc_grouped_wgrad(p[0], p[1], P(256), None, None, 2, 4, 4, 4, c, c, dt, p[2], None, P(256), 1 << 40, None)

    f32, f16, bf16 = 0, 1, 2
    for shift, c, dt in ((8, 8, f16), (8, 64, bf16), (4, 8, f32), (8, 4, f32), (4, 4, f16), (2, 12, bf16), (2, 33, f32),
                         (1, 33, f16), (3, 5, bf16)):
        assert set(codes(shift, c, dt)) == {1}, (shift, c, dt)
