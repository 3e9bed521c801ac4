"""CPU checks of the norm, the 4-bit products and the page calls: exported symbols, the quantizer's and the packer's bytes
against the oracle, and every argument error, reported before anything would reach a GPU."""
import ctypes
import os
import re
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from oracle import step_oracle as S  # noqa: E402

P = 4096                                       # an aligned address; refused calls touch no memory


@pytest.fixture(scope="module")
def q():
    import torch  # noqa: F401
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


def test_header_symbols_exported(q):
    src = open(os.path.join(ROOT, "include", "qmoe_step.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", src)))
    lib = ctypes.CDLL(q.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    assert sorted(q.EXPORTED_STEP) == names and len(names) == 10


# ---------------------------------------------------------------------------
# Quantizer and packer.

SHAPES = [(1, 8, 32), (16, 128, 128), (17, 136, 64), (5, 40, 128), (33, 392, 32), (48, 1024, 128)]


def _weights(rng, n, k):
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    w[0, : k // 2] = np.abs(w[0, : k // 2])        # one-sided groups, zeros, a wide one
    w[n // 2] = 0
    w[-1] *= 1000
    return w


@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_and_pack(q, n, k, group, zeros):
    w = _weights(np.random.default_rng(n + k), n, k)
    codes, scales, zp = q.moe_linear_quantize(w, group, zeros, n_threads=3)
    oc, os_, oz = S.quantize4(w, group, zeros)
    assert np.array_equal(codes, oc) and np.array_equal(scales.astype(np.float64), os_)
    assert (zp is None) != zeros and (zp is None or np.array_equal(zp, oz))
    for threads in (1, 5):
        packed = q.moe_linear_pack(codes, scales, zp, group, n_threads=threads)
        assert packed.size == q.moe_linear_packed_bytes(n, k, group, zeros)
        assert np.array_equal(packed, S.pack4(oc, os_, oz if zeros else None, group))
    # half a step of the weights at most, where neither end cuts off (the zero point, and the scale, are rounded too)
    back = S.weights4(codes, scales, np.full(oz.shape, 8) if zp is None else zp, group)
    step = np.repeat(scales.astype(np.float64), group, 1)[:, :k]
    assert np.all(np.abs(back - w) <= step * (1.0 if zeros else 0.5) * (1 + 2.0 ** -9) + step * 7 * 2.0 ** -10)


def test_pack_any_codes(q):
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (35, 264), dtype=np.uint8)
    scales = rng.integers(0, 0x7C00, (35, 5), dtype=np.uint16).view(np.float16)      # subnormal ones too
    scales[::2] *= -1
    zeros = rng.integers(0, 16, (35, 5), dtype=np.uint8)
    assert np.array_equal(q.moe_linear_pack(codes, scales, zeros, 64), S.pack4(codes, scales, zeros, 64))


def test_packing_refused(q):
    lib, e = q.lib, q.MOE_ERR_INVALID_ARG
    w, codes, s, z = np.zeros((4, 32), np.float32), np.zeros((4, 32), np.uint8), np.zeros((4, 1), np.uint16), np.zeros((4, 1), np.uint8)
    out = np.full(q.moe_linear_packed_bytes(4, 32, 32, True), 0xA5, np.uint8)
    a = lambda x: x.ctypes.data  # noqa: E731
    for n, k, g in ((0, 32, 32), (4, 0, 32), (4, 36, 32), (4, 32, 16), (4, 32, 0), (4, 32, 256), (-4, 32, 32), ((1 << 24) + 1, 32, 32),
                    (4, (1 << 20) + 8, 32)):
        assert q.lib.moe_linear_packed_bytes(n, k, g, 0) == 0
        assert lib.moe_linear_quantize(a(w), n, k, g, a(codes), a(s), None, 1) == e
        assert lib.moe_linear_pack(a(codes), a(s), None, n, k, g, a(out), out.nbytes, 1) == e and "moe_linear_pack" in q.moe_last_error()
    for args in ((None, 4, 32, 32, a(codes), a(s)), (a(w), 4, 32, 32, None, a(s)), (a(w), 4, 32, 32, a(codes), None)):
        assert lib.moe_linear_quantize(*args, None, 1) == e
    for bad in (np.nan, np.inf, 1e6):
        w[2, 5] = bad
        c2 = np.full_like(codes, 0xA5)
        assert lib.moe_linear_quantize(a(w), 4, 32, 32, a(c2), a(s), None, 1) == e and (c2 == 0xA5).all()
    assert lib.moe_linear_pack(None, a(s), None, 4, 32, 32, a(out), out.nbytes, 1) == e
    assert lib.moe_linear_pack(a(codes), None, None, 4, 32, 32, a(out), out.nbytes, 1) == e
    assert lib.moe_linear_pack(a(codes), a(s), None, 4, 32, 32, None, out.nbytes, 1) == e
    assert lib.moe_linear_pack(a(codes), a(s), a(z), 4, 32, 32, a(out), out.nbytes - 1, 1) == e
    codes[3, 31] = 16
    assert lib.moe_linear_pack(a(codes), a(s), None, 4, 32, 32, a(out), out.nbytes, 1) == e
    codes[3, 31], z[1, 0] = 15, 16
    assert lib.moe_linear_pack(a(codes), a(s), a(z), 4, 32, 32, a(out), out.nbytes, 1) == e
    z[1, 0], s[1, 0] = 15, 0xFC00
    assert lib.moe_linear_pack(a(codes), a(s), a(z), 4, 32, 32, a(out), out.nbytes, 1) == e
    assert (out == 0xA5).all()
    s[1, 0] = 0
    assert lib.moe_linear_pack(a(codes), a(s), a(z), 4, 32, 32, a(out), out.nbytes, 1) == 0 and q.moe_last_error() == ""


# ---------------------------------------------------------------------------
# Refusals.

def _norm(q, **kw):
    d = dict(rows=3, heads=2, cols=64, x_dtype=0, x=P, x_stride=128, residual_dtype=0, weight_dtype=2, residual=2 * P,
             residual_stride=128, sum=3 * P, sum_stride=128, weight=P, eps=1e-6, out_dtype=0, out=4 * P, out_stride=128, codes=5 * P,
             codes_stride=128, scales=P, scale_stride=4, group=0)
    d.update(kw)
    return q.lib.moe_rms_norm(ctypes.byref(q.MoeNorm(*d.values())), None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=(1 << 24) + 1), dict(heads=0), dict(heads=5000), dict(rows=1 << 23), dict(cols=0), dict(cols=12),
    dict(cols=16392), dict(x=None), dict(x=P + 8), dict(x_stride=120), dict(x_stride=132), dict(x_stride=(1 << 24) + 8), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(residual=P + 2), dict(residual_stride=64), dict(residual=None),
    dict(sum=P + 4), dict(sum_stride=0), dict(weight=P + 2), dict(out=P + 1), dict(out_stride=-128), dict(codes=None), dict(scales=None),
    dict(codes=5 * P + 8), dict(codes_stride=100), dict(scales=P + 4), dict(scale_stride=2), dict(scale_stride=6), dict(scale_stride=0),
    dict(out=None, codes=None, scales=None, sum=None), dict(out=3 * P), dict(codes=3 * P), dict(codes=4 * P),
    dict(sum=P, sum_stride=136), dict(sum=2 * P, sum_stride=136), dict(sum=P, x_dtype=1), dict(out=P, out_stride=256),
    dict(out=2 * P, out_dtype=1), dict(codes=P), dict(codes=2 * P)])
def test_norm_refused(q, kw):
    assert _norm(q, **kw) == q.MOE_ERR_INVALID_ARG and "moe_rms_norm" in q.moe_last_error()


@pytest.mark.parametrize("kw", [dict(x_dtype=3), dict(x_dtype=-1), dict(residual_dtype=3), dict(weight_dtype=4), dict(out_dtype=3), dict(group=64)])
def test_norm_unsupported(q, kw):
    assert _norm(q, **kw) == q.MOE_ERR_UNSUPPORTED


def test_nothing_to_do(q):
    assert _norm(q, rows=0) == q.MOE_OK
    assert q.lib.moe_rms_norm(None, None) == q.MOE_ERR_INVALID_ARG
    assert _linear(q, rows=0) == q.MOE_OK


def _linear(q, w={}, **kw):
    m = dict(n=48, k=256, group=64, with_zeros=0, packed=P, bias=P)
    m.update(w)
    d = dict(rows=3, x_dtype=3, x=P, x_stride=256, x_scales=P, scale_stride=4, x_group=128, y_dtype=2, y=2 * P, y_stride=48)
    d.update(kw)
    return q.lib.moe_linear(ctypes.byref(q.MoeLinearWeights(*m.values())), *d.values(), None)


@pytest.mark.parametrize("w,kw", [
    (dict(n=0), {}), (dict(k=252), {}), (dict(k=0), {}), (dict(group=48), {}), (dict(packed=None), {}), (dict(packed=P + 8), {}),
    (dict(bias=P + 2), {}), ({}, dict(rows=-1)), ({}, dict(rows=(1 << 20) + 1, scale_stride=1 << 21)), ({}, dict(x=None)), ({}, dict(x=P + 4)),
    ({}, dict(x_stride=248)), ({}, dict(x_stride=260)), ({}, dict(x_stride=(1 << 24) + 8)), ({}, dict(x_scales=None)),
    ({}, dict(x_scales=P + 8)), ({}, dict(scale_stride=0)), ({}, dict(scale_stride=5)), ({}, dict(rows=5)), ({}, dict(y=None)),
    ({}, dict(y=P + 8)), ({}, dict(y_stride=47)), ({}, dict(y_stride=(1 << 24) + 1)), ({}, dict(y=P)), ({}, dict(x_dtype=0)),
    ({}, dict(x_dtype=1, x_scales=None))])
def test_linear_refused(q, w, kw):
    assert _linear(q, w, **kw) == q.MOE_ERR_INVALID_ARG and "moe_linear" in q.moe_last_error()


@pytest.mark.parametrize("kw", [dict(x_dtype=2), dict(x_dtype=9), dict(y_dtype=3), dict(y_dtype=-1), dict(x_group=64)])
def test_linear_unsupported(q, kw):
    assert _linear(q, **kw) == q.MOE_ERR_UNSUPPORTED


def _page_calls(q, pool={}, tables={}, cache={}, n_caches=2, ws_bytes=1 << 40, ws=P, lens=2 * P, out=P):
    c = dict(n_pages=64, page_tokens=32, kv_heads=2, head_dim=64, codes=P, scales=P)
    c.update(cache)
    p = dict(n_pages=64, n_caches=n_caches, caches=(q.MoeKvCache * 2)(q.MoeKvCache(*c.values()), q.MoeKvCache(*c.values())), refs=P)
    p.update(pool)
    t = dict(seqs=8, pages_per_seq=4, page_tokens=32, page_table=P, table_stride=4, kv_lens=P)
    t.update(tables)
    a = q.MoeKvPool(*p.values()), q.MoeKvTables(*t.values())
    R, lib = ctypes.byref, q.lib
    return a, [lambda: lib.moe_kv_resize(R(a[0]), R(a[1]), lens, out, None),
               lambda: lib.moe_kv_fork(R(a[0]), R(a[1]), lens, out, ws, ws_bytes, None),
               lambda: lib.moe_kv_compact(R(a[0]), R(a[1]), out, ws, ws_bytes, None)]


BAD_PAGES = [dict(pool=dict(n_pages=0)), dict(pool=dict(n_pages=(1 << 30) + 1)), dict(pool=dict(n_caches=-1)), dict(pool=dict(n_caches=257)),
             dict(pool=dict(caches=None)), dict(pool=dict(refs=None)), dict(pool=dict(refs=P + 8)), dict(pool=dict(n_pages=63)),
             dict(tables=dict(seqs=0)), dict(tables=dict(seqs=4097)), dict(tables=dict(pages_per_seq=0)), dict(tables=dict(page_tokens=24)),
             dict(tables=dict(page_tokens=8)), dict(tables=dict(page_tokens=2048)), dict(tables=dict(page_tokens=64)),
             dict(tables=dict(page_table=None)), dict(tables=dict(page_table=P + 2)), dict(tables=dict(kv_lens=None)), dict(tables=dict(kv_lens=P + 1)),
             dict(tables=dict(table_stride=3)), dict(tables=dict(pages_per_seq=1 << 26, table_stride=1 << 26)),
             dict(tables=dict(seqs=4096, pages_per_seq=1 << 19, table_stride=1 << 19)), dict(cache=dict(kv_heads=0)),
             dict(cache=dict(head_dim=96)), dict(cache=dict(codes=None)), dict(cache=dict(codes=P + 8)), dict(cache=dict(scales=None)),
             dict(cache=dict(scales=P + 2))]


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_pages_refused(q, kw):
    (pool, tables), calls = _page_calls(q, **kw)
    for call in calls:
        assert call() == q.MOE_ERR_INVALID_ARG and "moe_kv_" in q.moe_last_error()
    for f in (q.lib.moe_kv_fork_workspace_bytes, q.lib.moe_kv_compact_workspace_bytes):
        assert f(ctypes.byref(pool), ctypes.byref(tables)) == 0


def test_page_arguments_refused(q):
    for kw, which in ((dict(lens=None), (0, 1)), (dict(lens=P + 2), (0, 1)), (dict(out=P + 1), (0, 1, 2)), (dict(ws=None), (1, 2)),
                      (dict(ws=P + 8), (1, 2)), (dict(lens=P), (0,))):
        calls = _page_calls(q, **kw)[1]
        for i in which:
            assert calls[i]() == q.MOE_ERR_INVALID_ARG, (kw, i)
    (pool, tables), _ = _page_calls(q)
    R = ctypes.byref
    for f, i in ((q.lib.moe_kv_fork_workspace_bytes, 1), (q.lib.moe_kv_compact_workspace_bytes, 2)):
        need = f(R(pool), R(tables))
        assert need > 0 and _page_calls(q, ws_bytes=need - 1)[1][i]() == q.MOE_ERR_WORKSPACE and str(need) in q.moe_last_error()
    assert q.lib.moe_kv_resize(None, R(tables), P, None, None) == q.MOE_ERR_INVALID_ARG
    assert q.lib.moe_kv_resize(R(pool), None, P, None, None) == q.MOE_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(q):
    import torch
    x = torch.zeros((2, 64))
    q_device, q._device = q._device, lambda: 0
    try:
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            q.moe_rms_norm(x, x, stream=0)
    finally:
        q._device = q_device
    with pytest.raises(ValueError, match="packed must be a CUDA tensor"):
        q.LinearWeights(torch.zeros(4096, dtype=torch.uint8), 16, 128)
    with pytest.raises(ValueError, match="group"):
        q.LinearWeights(torch.zeros(4096, dtype=torch.uint8), 16, 128, group=16)
    with pytest.raises(ValueError, match="refs must be a CUDA tensor"):
        q.KvPool(torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="page_table"):
        q.KvTables(torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="scales and zeros"):
        q.moe_linear_pack(np.zeros((4, 64), np.uint8), np.zeros((4, 1), np.float16), None, 32)


def test_scales_shape(q):
    assert q.moe_scales_shape(5, 300, 128) == (3, 8) and q.moe_scales_shape(4, 300) == (1, 4) and q.moe_scales_shape(1, 64, 128, 6) == (6, 4)
