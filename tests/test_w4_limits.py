"""Calls of the layer's operators at the limits of their sizes and without an operand, on the CPU."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)
NONE = ctypes.c_void_p(None)


@pytest.fixture(scope="module")
def cq():
    from minimax_scale_search_b200 import build
    build.build()
    from minimax_scale_search_b200 import cq as binding
    return binding


@pytest.mark.parametrize("R", [(1 << 31) - 8, (1 << 31) - 120])
def test_outputs_whose_last_tile_passes_31_bits_are_refused(cq, R):
    """The last tile of 128 outputs would end at 2^31, which 32-bit tile coordinates do not reach."""
    assert cq.lib.cq_w4_linear_backward(FAKE, R, FAKE, 128, 0, 4, FAKE, FAKE, FAKE, R, 128, FAKE, 128, FAKE, NONE) == \
        cq.CQ_ERR_UNSUPPORTED
    assert cq.lib.cq_w4_linear(FAKE, 128, 0, 40, FAKE, FAKE, FAKE, R, 128, NONE, 0, NONE, 0, FAKE, R, NONE, 0, NONE) == \
        cq.CQ_ERR_UNSUPPORTED
