"""CPU checks of the step calls' limits on sizes, each one past the limit with all else in order, and each at the limit with
another fault that is looked at later."""
import pytest

from test_step_host import P, _norm, q  # noqa: F401

MANY = dict(codes=None, scales=None, heads=1, x_stride=16384, residual_stride=16384, sum_stride=16384, out_stride=16384)


@pytest.mark.parametrize("cols,heads,most", [(64, 1, (1 << 24) - 1), (512, 3, ((1 << 24) - 1) // 3), (2048, 1, (1 << 24) - 1),
                                             (2056, 1, (1 << 23) - 1), (4096, 2, (1 << 22) - 1), (4104, 1, (1 << 22) - 1),
                                             (16384, 1, (1 << 22) - 1), (8, 4096, 4095)])
def test_norm_rows(q, cols, heads, most):  # noqa: F811
    kw = dict(MANY, cols=cols, heads=heads)
    for name in ("x_stride", "residual_stride", "sum_stride", "out_stride"):
        kw[name] = cols * heads
    assert _norm(q, rows=most + 1, **kw) == q.MOE_ERR_INVALID_ARG and "rows" in q.moe_last_error()
    assert _norm(q, rows=most, **dict(kw, x=None)) == q.MOE_ERR_INVALID_ARG and "x is NULL" in q.moe_last_error()
