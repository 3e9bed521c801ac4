"""GPU parity of moe_linear's split of 8-bit rows over workgroups that groups of 32 columns take beyond some 28700 weight rows
(4 weight tiles for up to 8 rows)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

from test_gpu_step_linear import run  # noqa: E402


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


@pytest.mark.parametrize("rows,n", [(1, 28721), (8, 32001)])
@pytest.mark.parametrize("zeros,x_group", [(False, 0), (False, 128), (True, 0), (True, 128)])
def test_wide_with_groups_of_32(q, rows, n, zeros, x_group):
    run(q, np.random.default_rng(rows + n), n, 328, rows, "int8", 32, zeros, "fp32", True, x_group, (8, 3))
