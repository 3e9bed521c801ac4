"""CPU checks of the step calls' limits on sizes, each one past the limit with all else in order, and each at the limit with
another fault that is looked at later; and of values that a cast would change."""
import ctypes

import numpy as np
import pytest

from test_step_host import _norm, _page_calls, q  # noqa: F401

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


@pytest.mark.parametrize("bad", [np.int64(256), np.int32(-256), np.uint16(512 + 7), np.int64(16), np.int8(-1), np.float32(7.5), np.float64("nan"),
                                 np.float32("inf"), np.float64(-0.25)])
def test_pack_refuses_what_bytes_do_not_hold(q, bad):  # noqa: F811
    """Codes and zero points of other types come as they are or not at all."""
    scales = np.ones((4, 2), np.float16)
    for name in ("codes", "zeros"):
        a = dict(codes=np.full((4, 64), 3, bad.dtype), zeros=np.full((4, 2), 5, bad.dtype))
        fine = q.moe_linear_pack(a["codes"], scales, a["zeros"], 32)
        assert np.array_equal(fine, q.moe_linear_pack(a["codes"].astype(np.uint8), scales, a["zeros"].astype(np.uint8), 32))
        a[name][2, 1] = bad
        with pytest.raises((ValueError, q.QmoeError)):
            q.moe_linear_pack(a["codes"], scales, a["zeros"], 32)


def test_most_pages(q):  # noqa: F811
    """2^29 pages are a pool, one more is none, with nothing else that could be wrong."""
    for f in (q.lib.moe_kv_fork_workspace_bytes, q.lib.moe_kv_compact_workspace_bytes):
        for n, fine in (((1 << 29), True), ((1 << 29) + 1, False), (1, True), (0, False)):
            (pool, tables), calls = _page_calls(q, pool=dict(n_pages=n, caches=None), n_caches=0)
            pool.n_caches = 0
            assert (f(ctypes.byref(pool), ctypes.byref(tables)) > 0) == fine, n
            if not fine:
                for call in calls:
                    assert call() == q.MOE_ERR_INVALID_ARG and "n_pages" in q.moe_last_error()
