"""CPU checks: arguments of the attention calls that are refused before anything would reach a GPU."""
import ctypes

import numpy as np
import pytest

P = 4096                                       # an aligned address; refused calls touch no memory


@pytest.fixture(scope="module")
def q():
    import torch  # noqa: F401
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


@pytest.mark.parametrize("scale", [float(np.finfo(np.float32).max), 2.4e38])
def test_scales_whose_factor_is_infinite(q, scale):
    """Scores are multiplied by scale * log2(e): an infinite one makes not a number of a score of zero."""
    R, lib = ctypes.byref, q.lib
    cache = q.MoeKvCache(8, 64, 2, 64, P, P)
    batch = q.MoeKvBatch(2, 6, 3, 4, P, 4, P, None)
    packed = q.MoePacked(2, 8, 8, 4, P, P, 4, 2, 64)
    calls = [lambda: lib.moe_attn_decode(R(cache), R(batch), 0, P, 256, 4, scale, 2 * P, 256, None, P, 0, None),
             lambda: lib.moe_attn_prefill(R(packed), 0, P, 256, P, 128, P, 128, scale, 1, 2 * P, 256, None, P, 0, None)]
    for call in calls:                         # (without a workspace: no call could get to a kernel)
        assert call() == q.MOE_ERR_INVALID_ARG and "scale" in q.moe_last_error()
