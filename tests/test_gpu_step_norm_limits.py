"""GPU checks of moe_rms_norm against the 64-bit oracle where a code is exactly between two whole numbers, and
where a root is not one of the 32-bit numbers."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

from attn_fixture import f64  # noqa: E402
from oracle import step_oracle as S  # noqa: E402
from test_gpu_step_norm import check_out, run  # noqa: E402


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


# Whole numbers whose 64-bit reciprocals are rounded, ones whose are not, and one scaled far from 1.
SCALES = [1, 3, 49, 98, 103, 107, 161, 197, 256, 49 * 2.0 ** -40]


@pytest.mark.parametrize("cols", [8, 64, 392, 512, 2056, 7168, 12296])
@pytest.mark.parametrize("size", [1.0, 49.0, 3 * 2.0 ** -20])
def test_codes_on_borders(q, cols, size):
    """Rows of +-size, whose root mean square is size: y is the weight, and the weights are halves of the scale.  The even
    neighbour is the code."""
    rng = np.random.default_rng(cols)
    for scale in SCALES:
        for group in (0, 128):
            half = rng.integers(-127, 127, cols) + 0.5
            half[::group or cols] = 127
            w = half * scale
            x = size * rng.choice([-1.0, 1.0], (2, cols))
            assert np.array_equal(w.astype(np.float32), w) and np.array_equal(x.astype(np.float32), x)
            xd, wd = torch.from_numpy(x).float().cuda(), torch.from_numpy(w).float().cuda()
            cd = torch.empty((2, cols), dtype=torch.int8, device="cuda")
            sc = torch.empty(q.moe_scales_shape(2, cols, group), device="cuda")
            q.moe_rms_norm(xd, None, wd, 0.0, codes=cd, scales=sc, group=group)
            codes, scales = S.codes8(S.rms_norm(x, w, 0.0), group)
            assert (scales == np.float32(scale)).all() and np.array_equal(codes, np.sign(x) * np.rint(half))
            assert np.array_equal(f64(sc)[:, :2], scales.T), scale
            got = cd.cpu().numpy()
            assert np.array_equal(got, codes), (scale, group, np.argwhere(got != codes)[:4].tolist())


@pytest.mark.parametrize("cols", [8, 64, 264, 2048, 7168, 16384])
def test_smallest_and_largest_values(q, cols):
    """Roots below 2^-126 and above 2^127: values below the normal numbers without epsilon, rows of nearly the largest one."""
    rng = np.random.default_rng(cols)
    sign = rng.choice([-1.0, 1.0], (10, cols))
    x = np.ones((10, cols))
    x[0] = 1e-39
    x[1] = 2.0 ** -149                                  # the smallest number
    x[2] = 2.0 ** -133                                  # the smallest bf16
    x[3] = 1e-40 * np.abs(rng.standard_normal(cols))
    x[4, :-1], x[4, -1] = 0, 1e-41
    x[5] = 2.0 ** -127
    x[6] = 3.3e38
    x[7] = 2.0 ** 126
    x[8] = 2.0 ** 127 * (1 - 2.0 ** -8)
    x[9] = 3.38e38 * rng.random(cols)
    for group in (None, 0, 128):
        for ot, wt in (("fp32", "bf16"), ("bf16", None), ("fp16", "fp32")):
            run(q, rng, 10, 1, cols, "fp32", None, ot, wt, group, x=x * sign, eps=0.0, what=f"fp32 {ot} {wt} {group}")
            run(q, rng, 10, 1, cols, "bf16", None, ot, wt, group, x=x * sign, eps=0.0, what=f"bf16 {ot} {wt} {group}")
            run(q, rng, 10, 1, cols, "bf16", "fp32", ot, wt, group, x=np.zeros_like(x), res=x * sign, eps=0.0, what=f"sum {ot} {wt} {group}")
            run(q, rng, 10, 1, cols, "fp32", None, ot, wt, group, x=x * sign, eps=1e-6, what=f"eps {ot} {wt} {group}")


@pytest.mark.parametrize("rows,cols", [((1 << 22) - 1, 4104), ((1 << 23) - 1, 2056)])
def test_most_rows(q, rows, cols):
    """As many vectors as the call takes, in place; rows at both ends and around 2^32 elements against the oracle."""
    rng = np.random.default_rng(cols)
    block = torch.from_numpy(rng.standard_normal((64, cols))).bfloat16().cuda()
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    at = [0, 1, (1 << 32) // cols - 1, (1 << 32) // cols, (1 << 32) // cols + 1, rows - 2, rows - 1]
    for i, r in enumerate(at):
        x[r] = block[i]
    q.moe_rms_norm(x, x, None, 0.0)
    for i, r in enumerate(at):
        check_out(x[r], S.rms_norm(f64(block[i]), 1.0, 0.0), torch.bfloat16, f"row {r}")
    x[at[0]:at[1] + 1], x[at[2]:at[4] + 1], x[at[5]:] = 1.0, 1.0, 1.0
    assert bool((x == 1.0).all())
