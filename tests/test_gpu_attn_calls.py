"""GPU tests of calls to the attention entry points that their header allows: drafts that are cut back, lengths and row
offsets outside of their range, far positions code by code, packed prompts without row offsets."""
import ctypes

import numpy as np
import pytest

from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    assert torch.cuda.is_available(), "GPU test needs a GPU"
    from bit_quantized_moe_02_amd import qmoe
    return qmoe


import torch  # noqa: E402

from attn_fixture import DT, attention_bounds, check_attention, cu_of, f64, i32, page_table, random_cache, rounded, rows_in, to_device  # noqa: E402


def _same(dev, ref):
    got = A.Cache(dev.codes.cpu().numpy(), f64(dev.scales), ref.page, ref.heads, ref.dim)
    assert np.array_equal(got.scales, ref.scales)
    assert np.array_equal(got.codes[:, :, :, 1], ref.codes[:, :, :, 1]), "V codes differ"
    assert np.array_equal(got.codes[:, :, :, 0], ref.codes[:, :, :, 0]), "K codes differ"


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_after_a_draft_is_cut_back(q, dt):
    """A rejected draft's large values: the block keeps their scale, and its kept tokens the second rounding, until its
    first slot is written again; a block that only the draft was in starts anew."""
    dt = DT[dt]
    rng = np.random.default_rng(70)
    D, Hk, page = 64, 2, 16
    table, n_pages = page_table(rng, [64], page)
    codes, scales = random_cache(rng, n_pages, page, Hk, D)
    ref = A.Cache(codes, scales, page, Hk, D)
    dev = to_device(q, ref)

    def step(first, n, sigma):
        kt, kv = rows_in(rng, n, Hk, D, dt, sigma=sigma)
        vt, vv = rows_in(rng, n, Hk, D, dt, sigma=sigma)
        q.moe_kv_append(dev, q.KvBatch(i32(table), i32([first + n]), n), kt, vt)
        ref.append(table[0], first, kv, vv)
        _same(dev, ref)
        return np.abs(kv).max((0, 2))

    def scale(pos):
        page_, blk = ref.block(table[0], pos)
        return ref.scales[page_, :, blk, 0]

    small = step(0, 12, 2.0 ** -10)                     # a prompt of small values
    step(12, 8, 64.0)                                   # a draft over two blocks, rejected
    step(12, 2, 2.0 ** -10)
    assert np.all(scale(0) > 2.0 ** 10 * small / 448)   # the block's scale is still the draft's
    step(14, 6, 2.0 ** -10)
    assert np.all(scale(16) < 2.0 ** -10)               # the next block's first slot was written again
    step(0, 12, 2.0 ** -10)
    assert np.all(scale(0) < 2.0 ** -10)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_read_and_append_clamp_lengths(q, dt):
    """Lengths below zero and behind the page table, row offsets behind the rows: the same rows and codes as with the
    values in their range, and nothing outside of the buffers."""
    dt = DT[dt]
    rng = np.random.default_rng(71)
    Hk, D, page, guard = 1, 64, 16, 4096
    table, n_pages = page_table(rng, [32, 32, 32], page)
    ref = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    codes = torch.full((ref.codes.size + 2 * guard,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((ref.scales.size + 2 * guard,), 77.0, device="cuda")
    codes[guard:-guard] = torch.from_numpy(ref.codes.reshape(-1)).cuda()
    scales[guard:-guard] = torch.from_numpy(ref.scales.astype(np.float32).reshape(-1)).cuda()
    dev = q.KvCache(codes[guard:-guard], scales[guard:-guard], page, Hk, D)
    batch = q.KvBatch(i32(table), i32([32, -5, 1 << 30]), 4, 2, i32([0, 1, 2, 77]))
    back = [torch.full((8, Hk, D), 5.0, dtype=dt, device="cuda") for _ in range(2)]
    q.moe_kv_read(dev, batch, back[0][2:6], back[1][2:6])
    torch.cuda.synchronize()
    for part, got in enumerate(back):
        assert torch.all(got[:2] == 5.0) and torch.all(got[6:] == 5.0)
        got = f64(got[2:6])
        assert np.array_equal(got[0], ref.read(table[0], 31, 32)[part][0])
        assert np.all(got[1] == 0)                      # (a position below zero)
        assert np.array_equal(got[2:], ref.read(table[2], 30, 32)[part])

    kt, kv = rows_in(rng, 4, Hk, D, dt)
    vt, vv = rows_in(rng, 4, Hk, D, dt)
    k_out = torch.full((8, Hk, D), 5.0, dtype=dt, device="cuda")
    q.moe_kv_append(dev, batch, kt, vt, k_out=k_out[2:6])
    torch.cuda.synchronize()
    ref.append(table[0], 31, kv[:1], vv[:1])
    ref.append(table[2], 30, kv[2:], vv[2:])
    _same(dev, ref)
    assert torch.equal(k_out[2:6], kt) and torch.all(k_out[:2] == 5.0) and torch.all(k_out[6:] == 5.0)
    for buf, fill in ((codes, 0x55), (scales, 77.0)):
        assert torch.all(buf[:guard] == fill) and torch.all(buf[-guard:] == fill), "written outside of the cache"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_far_positions_code_by_code(q, dt, inter):
    """k rows, K codes and scales near position 2^20 equal 64-bit arithmetic's."""
    dt = DT[dt]
    rng = np.random.default_rng(72)
    D, Hk, page, n = 128, 2, 1024, 40
    L = (1 << 20) - 3
    table = np.full((1, 1024), -1, np.int64)
    table[0, L // page] = 1
    ref = A.Cache(*random_cache(rng, 2, page, Hk, D), page, Hk, D)
    dev = to_device(q, ref)
    kt, kv = rows_in(rng, n, Hk, D, dt)
    vt, vv = rows_in(rng, n, Hk, D, dt)
    k_out = torch.zeros_like(kt)
    freqs = q.moe_rope_freqs(D)
    q.moe_kv_append(dev, q.KvBatch(i32(table), i32([L]), n), kt, vt, q.Rope(torch.from_numpy(freqs).cuda(), D, inter, 1.25), k_out=k_out)
    want = A.rotate(kv, np.arange(L - n, L), freqs, inter, 1.25)
    assert np.array_equal(f64(k_out), rounded(want, dt))
    ref.append(table[0], L - n, want, vv)
    _same(dev, ref)


@pytest.mark.parametrize("width", [1040, 1296, 1536, 1552])
@pytest.mark.parametrize("B", [1, 16])
def test_decode_by_the_tables_width(q, B, width):
    """Contexts next to where they are taken whole and where they are cut, few sequences and many, and a narrower view of
    a wide table: each right."""
    rng = np.random.default_rng(74)
    Hq, Hk, D, page, dt = 4, 2, 64, 16, torch.bfloat16
    lens = [1030] + [int(x) for x in rng.integers(0, 1030, B - 1)]
    table, n_pages = page_table(rng, lens, page, width=width // page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    dev = to_device(q, cache)
    qt, qv = rows_in(rng, B, Hq, D, dt, sigma=2.0)
    wide = torch.full((B, 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, :width // page] = i32(table)
    got = []
    for t in (i32(table), wide[:, :width // page], wide):
        batch = q.KvBatch(t, i32(lens), B)
        out, lse = torch.full_like(qt, 9.0), torch.full((B, Hq), 9.0, device="cuda")
        ws = torch.full((q.moe_attn_decode_workspace_bytes(dev, batch, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
        q.moe_attn_decode(dev, batch, qt, out, ws, D ** -0.5, lse)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for b, length in enumerate(lens):
        K, V, _ = cache.read(table[b], 0, length)
        ref, rl, mag, smag = A.attention(qv[b:b + 1], K, V, np.ones((1, length), bool), D ** -0.5)
        bounds = attention_bounds(dt, D, V, ref, mag, smag, length)
        for out, lse in got[1:]:
            check_attention(out[b:b + 1], lse[b:b + 1], ref, rl, *bounds, f"sequence {b}")


@pytest.mark.parametrize("n_keys", [60, 6000])          # whole, and cut into parts
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_without_row_offsets(q, D, dt, n_keys):
    """cu_q, cu_k or both NULL: the bits of the call with the same rows each."""
    dt = DT[dt]
    rng = np.random.default_rng(73)
    B, Hq, Hk, nq = 3, 4, 2, 21
    Tq, Tk = B * nq, B * n_keys
    x, k, v = (rows_in(rng, n, h, D, dt, pad=8)[0] for n, h in ((Tq, Hq), (Tk, Hk), (Tk, Hk)))
    cu_q, cu_k = i32(cu_of([nq] * B)), i32(cu_of([n_keys] * B))
    got = []
    for a, b in ((cu_q, cu_k), (None, cu_k), (cu_q, None), (None, None)):
        p = q.MoePacked(B, Tq, Tk, nq, None if a is None else a.data_ptr(), None if b is None else b.data_ptr(), Hq, Hk, D)
        need = q.lib.moe_attn_prefill_workspace_bytes(ctypes.byref(p))
        assert (need > 256) == (n_keys == 6000)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = torch.full((Tq, Hq, D), 9.0, dtype=dt, device="cuda"), torch.full((Tq, Hq), 9.0, device="cuda")
        rc = q.lib.moe_attn_prefill(ctypes.byref(p), q.MOE_DT_BF16 if dt == torch.bfloat16 else q.MOE_DT_F16, x.data_ptr(), x.stride(0),
                                    k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), D ** -0.5, 1, out.data_ptr(), out.stride(0),
                                    lse.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert rc == 0, q.moe_last_error()
        torch.cuda.synchronize()
        got.append((out, lse))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])
    kv, vv = f64(k)[:n_keys], f64(v)[:n_keys]
    seen = np.arange(n_keys)[None] <= (n_keys - nq + np.arange(nq))[:, None]
    ref, rl, mag, smag = A.attention(f64(x)[:nq], kv, vv, seen, D ** -0.5)
    check_attention(got[0][0][:nq], got[0][1][:nq], ref, rl, *attention_bounds(dt, D, vv, ref, mag, smag, n_keys), "first sequence")
