"""Sizes that a transformer block's layers take, and the first that they refuse (on the CPU: nothing is launched)."""

import ctypes

import pytest

import sparse_convolution_hash_gb300 as spc
from sparse_convolution_hash_gb300 import binding
from sparse_convolution_hash_gb300 import build as libbuild

UNSUPPORTED = 6
F16, BF16 = 1, 2
MOST_SEGMENTS = 1 << 30


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return binding.lib()


def p(v):
    return ctypes.c_void_p(v)


def test_attention_takes_as_many_segments_as_its_kernels_can_number(L):
    """Kernels look for a slot's segment with 32-bit steps: 32 of them, and the segment itself, stay below 2^31."""
    step = (MOST_SEGMENTS + 2 + 31) // 32
    assert MOST_SEGMENTS + 31 * step < 2 ** 31
    size = L.spc_attention_workspace_size
    assert size(4, 4, MOST_SEGMENTS, 1, 1, 8, F16, 1) > 0
    for segments in (MOST_SEGMENTS + 1, 2 ** 31 - 4, 2 ** 31 - 1):
        assert size(4, 4, segments, 1, 1, 8, F16, 1) == 0
        rows = [p(256), 8] * 3
        ends = [p(256), p(256), segments, 4, 4, 1, 1, 8, 0.5, BF16]
        assert L.spc_attention_fwd(*rows, *ends, p(1024), 8, p(2048), None, p(4096), 1 << 40, None) == UNSUPPORTED
        assert L.spc_attention_bwd(p(512), 8, *rows, p(1024), 8, p(2048), *ends, p(8192), 8, p(16384), 8, p(32768), 8, None, p(4096), 1 << 40,
                                   None) == UNSUPPORTED


@pytest.mark.parametrize("pairs", [(1.5, 2, 3), (2.0, 2, 2), ("1", 1, 1), (2 ** 32 + 1, 0, 0), (0, 0, 2 ** 31), (1, 2), (1, -2, 3)])
def test_rope_pairs_are_whole_numbers_of_32_bits(L, pairs):
    """A number's low half, or a fraction cut off, would be another call (also after calls with such whole numbers)."""
    assert len(spc.spc_rope_steps((2, 2, 2))) == 6 and len(spc.spc_rope_steps((1, 1, 1))) == 3
    with pytest.raises(ValueError):
        spc.spc_rope_steps(pairs)


@pytest.mark.parametrize("sizes,held", [((0, 0), True), ((7, 2 ** 31 - 1), True), ((-1, 5), False), ((2 ** 31, 1), False), ((8, 2 ** 32 + 8), False),
                                        ((-2 ** 32 + 8, 3), False)])
def test_sizes_that_32_bits_do_not_hold_are_refused(sizes, held):
    if held:
        return binding._held(sizes[0] | sizes[1], "here")
    with pytest.raises(spc.SpcError):
        binding._held(sizes[0] | sizes[1], "here")
