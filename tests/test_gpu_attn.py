"""GPU parity of the attention calls with the fp64 oracle: the cache's bytes,
rotated rows, rows read back, decode and prefill attention, at the sizes and
masks where they can go wrong, and a run of them together."""
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

from attn_fixture import (DT, attention_bounds, check_attention, cu_of, f64, half_step, i32, in_type, page_table, random_cache,  # noqa: E402
                          rounded, rows_in, spoil_tails, subnormal_half, to_device)


def _batch(q, table, lens, ns, uniform=False, pad_table=0):
    wide = np.full((len(lens), table.shape[1] + pad_table), -7, np.int64)
    wide[:, :table.shape[1]] = table
    t = i32(wide)[:, :table.shape[1]]
    return q.KvBatch(t, i32(lens), int(sum(ns)), max(max(ns), 1), None if uniform else i32(cu_of(ns)))


# ---------------------------------------------------------------------------
# append

APPEND = [  # new tokens, lengths after the step, page, rot, interleaved
    ([1], [1], 16, 64, False),
    ([1, 1, 1], [16, 17, 33], 16, 32, True),
    ([3, 1, 2, 5], [3, 1, 20, 100], 64, 64, False),
    ([40, 16, 7], [40, 57, 300], 32, 16, True),
    ([1, 4, 1], [0, 2, 31], 16, 64, False),          # an empty sequence; more rows than positions
    ([0, 5, 0], [9, 5, 0], 128, 0, False),            # sequences without rows
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(q, case, D, dt):
    ns, lens, page, rot, inter = APPEND[case]
    dt = DT[dt]
    rng = np.random.default_rng(100 + case)
    Hq, Hk = 5, 3
    rot = rot * D // 64
    table, n_pages = page_table(rng, lens, page)
    codes, scales = random_cache(rng, n_pages, page, Hk, D, sigma=0.25)
    cache = A.Cache(codes, scales, page, Hk, D)
    dev = to_device(q, cache)
    T = int(sum(ns)) + 2                                # two rows behind the last sequence
    qt, qv = rows_in(rng, T, Hq, D, dt, pad=24)
    kt, kv = rows_in(rng, T, Hk, D, dt, pad=8)
    vt, vv = rows_in(rng, T, Hk, D, dt)
    q_out = torch.full((T, Hq, D), 3.0, dtype=dt, device="cuda")
    k_out = torch.full((T, Hk + 1, D), 3.0, dtype=dt, device="cuda")[:, :Hk]
    batch = q.KvBatch(i32(table), i32(lens), T, max(ns), i32(cu_of(ns)))
    freqs = np.ascontiguousarray(q.moe_rope_freqs(max(rot, 16), 10000.0)[:rot // 2])
    rope = q.Rope(torch.from_numpy(freqs).cuda(), rot, inter, 1.25)
    q.moe_kv_append(dev, batch, kt, vt, rope, qt, q_out, k_out)
    torch.cuda.synchronize()

    cu = cu_of(ns)
    for name, x, got in (("q", qv, f64(q_out)), ("k", kv, f64(k_out))):
        assert np.all(got[cu[-1]:] == 3.0), f"{name}: rows behind the last sequence were written"
        for b, n in enumerate(ns):
            rows = slice(cu[b], cu[b + 1])
            pos = np.arange(lens[b] - n, lens[b])
            want = A.rotate(x[rows], pos, freqs, inter, 1.25) if rot else x[rows]
            # the turned value: three 32-bit operations and sines good to 2^-22 on |a| + |b|, then one rounding
            slack = 2.0 ** -20 * 1.25 * (2 * np.abs(x[rows]).max(initial=0)) if rot else 0.0
            tol = half_step(dt) * np.abs(want) + slack + subnormal_half(dt)
            assert np.all(np.abs(got[rows] - want) <= tol), (name, b, np.abs(got[rows] - want).max())
            if name == "k":
                assert np.array_equal(got[rows], rounded(want, dt)), (b, np.abs(got[rows] - want).max())

    # the cache, code by code: k is turned in 64 bits and rounded once, to its row type and to its codes
    ref = A.Cache(codes, scales, page, Hk, D)
    for b, n in enumerate(ns):
        pos = np.arange(lens[b] - n, lens[b])
        k = A.rotate(kv[cu[b]:cu[b + 1]], pos, freqs, inter, 1.25) if rot else kv[cu[b]:cu[b + 1]]
        ref.append(table[b], lens[b] - n, k, vv[cu[b]:cu[b + 1]])
    got = A.Cache(dev.codes.cpu().numpy(), f64(dev.scales), page, Hk, D)
    assert np.array_equal(got.scales, ref.scales)
    assert np.array_equal(got.codes[:, :, :, 1], ref.codes[:, :, :, 1]), "V codes differ"
    assert np.array_equal(got.codes[:, :, :, 0], ref.codes[:, :, :, 0]), "K codes differ"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 48), (128, 112), (256, 16), (256, 240)])
def test_append_turns_part_of_a_head(q, D, rot, inter):
    """Numbers of turned columns that are no power of two, over a border between blocks of a large page."""
    rng = np.random.default_rng(48)
    Hq, Hk, page, dt, lens, ns = 3, 1, 1024, torch.bfloat16, [1030, 18], [20, 5]
    table, n_pages = page_table(rng, lens, page)
    codes, scales = random_cache(rng, n_pages, page, Hk, D)
    dev = to_device(q, A.Cache(codes, scales, page, Hk, D))
    qt, qv = rows_in(rng, 25, Hq, D, dt)
    kt, kv = rows_in(rng, 25, Hk, D, dt)
    vt, _ = rows_in(rng, 25, Hk, D, dt)
    q_out, k_out = torch.full_like(qt, 3.0), torch.full_like(kt, 3.0)
    freqs = q.moe_rope_freqs(rot, 500.0, "base", 2.0)
    q.moe_kv_append(dev, _batch(q, table, lens, ns), kt, vt, q.Rope(torch.from_numpy(freqs).cuda(), rot, inter), qt, q_out, k_out)
    for x, got in ((qv, f64(q_out)), (kv, f64(k_out))):
        for b, rows in enumerate((slice(0, 20), slice(20, 25))):
            want = A.rotate(x[rows], np.arange(lens[b] - ns[b], lens[b]), freqs, inter)
            tol = half_step(dt) * np.abs(want) + 2.0 ** -20 * 2 * np.abs(x[rows]).max()
            assert np.all(np.abs(got[rows] - want) <= tol), np.abs(got[rows] - want).max()
            assert np.array_equal(got[rows][:, :, rot:], x[rows][:, :, rot:])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_token_by_token_equals_oracle(q, dt):
    """40 single-token steps whose values grow and shrink, V and unturned K: every byte equal, the growth of a block's
    scale and its earlier codes' second rounding included; zeros, infinities and NaN among them."""
    dt = DT[dt]
    D, Hk, page = 64, 2, 16
    rng = np.random.default_rng(7)
    table, n_pages = page_table(rng, [40, 40], page)
    codes, scales = random_cache(rng, n_pages, page, Hk, D, garbage=True)
    ref = A.Cache(codes, scales, page, Hk, D)
    dev = to_device(q, ref)
    for t in range(40):
        sigma = 2.0 ** ((t * 5) % 11 - 6)
        kt, kv = rows_in(rng, 2, Hk, D, dt, sigma=sigma)
        vt, vv = rows_in(rng, 2, Hk, D, dt, sigma=sigma * 0.3)
        if t % 7 == 3:
            vt[0, 1, 5], vt[1, 0, 63], kt[0, 0, 1] = float("inf"), float("nan"), -float("inf")
            kv, vv = f64(kt), f64(vt)
        if t % 9 == 4:
            vt[:] = 0
            vv = f64(vt)
        q.moe_kv_append(dev, _batch(q, table, [t + 1, t + 1], [1, 1], uniform=True), kt, vt)
        for b in (0, 1):
            ref.append(table[b], t, kv[b:b + 1], vv[b:b + 1])
    got, gs = dev.codes.cpu().numpy().reshape(ref.codes.shape), f64(dev.scales).reshape(ref.scales.shape)
    assert np.array_equal(gs, ref.scales, equal_nan=True)
    nan = (got & 0x7F) == 0x7F                          # either code for not a number
    assert np.array_equal(nan, (ref.codes & 0x7F) == 0x7F)
    assert np.array_equal(got[~nan], ref.codes[~nan])


def test_append_chunks_equal_one_call_where_the_scale_does_not_grow(q):
    """The same rows in one call or in odd pieces: the same bytes (the first token of each block holds its maximum)."""
    D, Hk, page, n = 128, 2, 64, 200
    rng = np.random.default_rng(8)
    table, n_pages = page_table(rng, [n], page)
    kt, kv = rows_in(rng, n, Hk, D, torch.bfloat16)
    vt, vv = rows_in(rng, n, Hk, D, torch.bfloat16)
    kt[::16, :, 0] = 30.0
    vt[::16, :, 0] = 30.0
    got = []
    for pieces in ([200], [1, 15, 16, 17, 3, 60, 88]):
        codes, scales = random_cache(np.random.default_rng(9), n_pages, page, Hk, D)
        dev = to_device(q, A.Cache(codes, scales, page, Hk, D))
        at = 0
        for p in pieces:
            q.moe_kv_append(dev, _batch(q, table, [at + p], [p]), kt[at:at + p], vt[at:at + p])
            at += p
        got.append((dev.codes.clone(), dev.scales.clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_append_in_place_far_positions_and_bad_pages(q):
    """q and k turned in place at positions near 2^20; pages that are none of the cache's get nothing."""
    D, Hk, Hq, page = 128, 2, 2, 1024
    rng = np.random.default_rng(10)
    L = (1 << 20) - 3
    table = np.full((2, 1024), -1, np.int64)
    table[0, L // page] = 0
    table[1, 0] = 99                                    # behind the cache's pages
    codes, scales = random_cache(rng, 2, page, Hk, D)
    ref = A.Cache(codes, scales, page, Hk, D)
    dev = to_device(q, ref)
    qkv = torch.from_numpy(rng.standard_normal((6, Hq + 2 * Hk, D))).to(torch.float16).cuda()
    x = f64(qkv)
    freqs = q.moe_rope_freqs(D)
    rope = q.Rope(torch.from_numpy(freqs).cuda(), D)
    qs, ks, vs = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    lens, ns = [L, 4], [3, 3]
    q.moe_kv_append(dev, _batch(q, table, lens, ns, pad_table=3), ks, vs, rope, qs, qs, ks)
    y = f64(qkv)
    assert np.array_equal(y[:, Hq + Hk:], x[:, Hq + Hk:])
    for b in (0, 1):
        pos = np.arange(lens[b] - 3, lens[b])
        want = A.rotate(x[3 * b:3 * b + 3, :Hq + Hk], pos, freqs)
        assert np.all(np.abs(y[3 * b:3 * b + 3, :Hq + Hk] - want) <= half_step(torch.float16) * np.abs(want) + 2.0 ** -20 * 8)
    got = dev.codes.cpu().numpy().reshape(ref.codes.shape)
    ref.append(table[0], L - 3, A.rotate(x[:3, Hq:Hq + Hk], np.arange(L - 3, L), freqs), x[:3, Hq + Hk:])
    assert np.array_equal(got[1], codes[1]), "a page nobody names was written"
    assert np.array_equal(got[0][:, :, 1], ref.codes[0][:, :, 1])


# ---------------------------------------------------------------------------
# read


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_read(q, page, D, dt):
    dt = DT[dt]
    rng = np.random.default_rng(20)
    lens, ns, Hk = [40, 0, 17, 16, 130], [40, 1, 5, 16, 99], 3
    table, n_pages = page_table(rng, lens, page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    table[4, 0] = n_pages + 5                           # a page of no tokens, in the middle of what is read for small pages
    dev = to_device(q, cache)
    T = sum(ns) + 1
    out = [torch.full((T, Hk * D + 8), 5.0, dtype=dt, device="cuda")[:, :Hk * D].unflatten(1, (Hk, D)) for _ in range(2)]
    q.moe_kv_read(dev, q.KvBatch(i32(table), i32(lens), T, max(ns), i32(cu_of(ns))), *out)
    got = [f64(o) for o in out]
    cu = cu_of(ns)
    for b, n in enumerate(ns):
        K, V, _ = cache.read(table[b], lens[b] - n, lens[b])
        for g, w in zip(got, (K, V)):
            assert np.array_equal(g[cu[b]:cu[b + 1]], in_type(w, dt)), b
    for g in got:
        assert np.all(g[cu[-1]:] == 5.0)


# ---------------------------------------------------------------------------
# decode


def _decode(q, cache, dev, table, lens, ns, Hq, dt, rng, what, uniform=False, sigma=1.0, extra=0, pad=0, check=True, spoil=None):
    D, Hk = cache.dim, cache.heads
    T = int(sum(ns)) + extra
    qt, qv = rows_in(rng, T, Hq, D, dt, pad=pad, sigma=sigma)
    if extra == 0:
        batch = _batch(q, table, lens, ns, uniform, pad_table=1)
    else:
        batch = q.KvBatch(i32(table), i32(lens), T, max(max(ns), 1), i32(cu_of(ns)))
    out = torch.full((T, Hq * D + pad), 9.0, dtype=dt, device="cuda")[:, :Hq * D].unflatten(1, (Hq, D))
    lse = torch.full((T, Hq), 9.0, device="cuda")
    ws = torch.full((q.moe_attn_decode_workspace_bytes(dev, batch, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    scale = D ** -0.5
    q.moe_attn_decode(dev, batch, qt, out, ws, scale, lse)
    torch.cuda.synchronize()
    if check:
        cu = cu_of(ns)
        assert torch.all(out[cu[-1]:] == 9.0) and torch.all(lse[cu[-1]:] == 9.0)
        for b, n in enumerate(ns):
            if n == 0:
                continue
            K, V, there = cache.read(table[b], 0, lens[b])
            K, V = in_type(K, dt), in_type(V, dt)
            seen = (np.arange(lens[b])[None] <= (lens[b] - n + np.arange(n))[:, None]) & there[None]
            rows = slice(cu[b], cu[b + 1])
            ref, rl, mag, smag = A.attention(qv[rows], K, V, seen, scale)
            tol, tl = attention_bounds(dt, D, V, ref, mag, smag, lens[b])
            check_attention(out[rows], lse[rows], ref, rl, tol, tl, f"{what}, sequence {b}")
    return qt, out, lse


DECODE = [  # rows, lengths, page, query heads, key heads
    ([1], [1], 16, 1, 1),
    ([1, 1, 1, 1, 1], [15, 16, 17, 31, 33], 16, 4, 2),
    ([1, 1, 1], [0, 700, 129], 64, 8, 1),
    ([3, 1, 2, 16], [3, 300, 1, 40], 32, 6, 2),        # a draft longer than its context
    ([16, 5], [16, 257], 16, 12, 3),                   # 64 rows of a key head
    ([16, 16], [100, 16], 128, 24, 2),                 # 192 rows: several row tiles
    ([33, 0, 1], [65, 5, 5], 64, 8, 1),                # more rows than a draft has
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(q, case, D, dt):
    ns, lens, page, Hq, Hk = DECODE[case]
    rng = np.random.default_rng(200 + case)
    table, n_pages = page_table(rng, lens, page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    spoil_tails(cache, table, lens)
    dev = to_device(q, cache)
    _decode(q, cache, dev, table, lens, ns, Hq, DT[dt], rng, f"case {case}", sigma=2.0, extra=2, pad=8)
    if len(set(ns)) == 1:
        _decode(q, cache, dev, table, lens, ns, Hq, DT[dt], rng, f"case {case}, uniform", uniform=True)


LONG = [  # rows, lengths, page, query heads, key heads: contexts cut into ranges
    ([1, 1, 1, 1], [3000, 1, 0, 1700], 64, 8, 2),
    ([4, 1, 0, 5, 2], [2100, 300, 9, 4, 1601], 16, 16, 2),             # two row tiles
    ([9, 3], [40, 2500], 128, 30, 3),                  # several workgroups of row tiles
    ([33, 1], [1999, 33], 32, 8, 1),                   # 264 rows of a key head
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(DECODE) + len(LONG)))
def test_decode_ranges(q, case, D, dt):
    """Page tables wide enough that contexts are cut into ranges, short contexts among them."""
    ns, lens, page, Hq, Hk = (DECODE + LONG)[case]
    rng = np.random.default_rng(260 + case)
    table, n_pages = page_table(rng, lens, page, width=4096 // page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    spoil_tails(cache, table, lens)
    dev = to_device(q, cache)
    _decode(q, cache, dev, table, lens, ns, Hq, DT[dt], rng, f"case {case}", sigma=2.0, extra=2, pad=8)


@pytest.mark.parametrize("width", [1, 40, 4000])
def test_decode_parts(q, width):
    """One context, page tables of several widths: from one part to one for each 128 positions, most of them empty."""
    rng = np.random.default_rng(30)
    Hk, D, page = 2, 128, 16
    lens = [16 * min(width, 40) - 3]
    table, n_pages = page_table(rng, lens, page, width=width)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    spoil_tails(cache, table, lens)
    _decode(q, cache, to_device(q, cache), table, lens, [2], 8, torch.bfloat16, rng, f"width {width}", sigma=3.0)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_decode_special_values(q, dt):
    """Values that are not numbers reach the rows that see their token and no other; peaked scores; a token of tiny V."""
    dt = DT[dt]
    rng = np.random.default_rng(31)
    Hk, D, page, lens, ns = 2, 64, 16, [70, 40], [5, 16]
    table, n_pages = page_table(rng, lens, page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    spoil_tails(cache, table, lens)
    for b, pos, part, h, d in ((0, 68, 1, 0, 3), (0, 69, 1, 1, 63), (1, 30, 1, 0, 17), (1, 35, 0, 1, 9), (1, 38, 1, 1, 40)):
        at = cache.block(table[b], pos)
        cache.codes[at[0], h, at[1], part, cache.at[part][pos % 16][d]] = 0xFF if d % 2 else 0x7F
    cache.scales[int(table[0, 1]), 1, 0, 1] = 2.0 ** -12
    _decode(q, cache, to_device(q, cache), table, lens, ns, 4, dt, rng, "special values", sigma=6.0)
    wide = np.concatenate([table, np.full((2, 200), -1)], axis=1)       # (the same cut into ranges)
    _decode(q, cache, to_device(q, cache), wide, lens, ns, 4, dt, rng, "special values, ranges", sigma=6.0)


@pytest.mark.parametrize("pad", [0, 60])
def test_decode_many_sequences(q, pad):
    """150 sequences of mixed lengths, empty slots and sequences without rows among them, so that ranges of the work
    begin and end anywhere; with wide page tables too."""
    rng = np.random.default_rng(43)
    Hk, D, page, B = 1, 64, 16, 150
    lens = [int(x) for x in rng.integers(0, 200, B)]
    lens[3], lens[70], lens[149] = 900, 0, 700
    ns = [int(x) for x in rng.integers(0, 3, B)]
    ns[3], ns[70], ns[149] = 2, 1, 1
    table, n_pages = page_table(rng, lens, page, width=57 + pad)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    spoil_tails(cache, table, lens)
    _decode(q, cache, to_device(q, cache), table, lens, ns, 2, torch.float16, rng, "many sequences", extra=1)


def test_decode_bad_pages(q):
    """Pages that are none of the cache's hold no tokens; a table of nothing else gives empty rows."""
    rng = np.random.default_rng(32)
    Hk, D, page, lens, ns = 1, 128, 16, [100, 50, 33], [1, 2, 1]
    table, n_pages = page_table(rng, lens, page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    table[0, 2], table[0, 6], table[1, :], table[2, 0] = -1, n_pages, 1 << 30, -(1 << 31)
    dev = to_device(q, cache)
    _, out, lse = _decode(q, cache, dev, table, lens, ns, 2, torch.bfloat16, rng, "bad pages")
    assert torch.all(out[1:3] == 0) and torch.all(lse[1:3] == -float("inf"))


def test_lengths_are_clamped(q):
    """Lengths below zero and behind the page table, row offsets behind the rows: nothing outside the buffers is touched,
    rows of the sequences in order are right."""
    rng = np.random.default_rng(33)
    Hk, D, page, Hq = 1, 64, 16, 2
    table, n_pages = page_table(rng, [32, 32, 32], page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    dev = to_device(q, cache)
    qt, qv = rows_in(rng, 4, Hq, D, torch.bfloat16)
    batch = q.KvBatch(i32(table), i32([32, -5, 1 << 30]), 4, 2, i32([0, 1, 2, 77]))
    ws = torch.empty(q.moe_attn_decode_workspace_bytes(dev, batch, Hq), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(qt), torch.zeros((4, Hq), device="cuda")
    q.moe_attn_decode(dev, batch, qt, out, ws, 0.125, lse)
    for b, length in ((0, 32), (2, 32)):
        rows = slice(0, 1) if b == 0 else slice(2, 4)
        n = rows.stop - rows.start
        K, V, _ = cache.read(table[b], 0, length)
        seen = np.arange(length)[None] <= (length - n + np.arange(n))[:, None]
        ref, rl, mag, smag = A.attention(qv[rows], K, V, seen, 0.125)
        check_attention(out[rows], lse[rows], ref, rl, *attention_bounds(torch.bfloat16, D, V, ref, mag, smag, length), f"sequence {b}")
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf"))
    back = torch.zeros((4, Hk, D), dtype=torch.bfloat16, device="cuda")
    q.moe_kv_read(dev, batch, back, back.clone())
    q.moe_kv_append(dev, batch, back, back)


def test_more_rows_than_max_new(q):
    """A sequence with more rows than max_new says: the first max_new are right, and nothing else is written."""
    rng = np.random.default_rng(44)
    Hk, D, page, Hq, lens, ns = 2, 128, 16, 2, [1500, 300], [9, 3]
    table, n_pages = page_table(rng, lens, page)
    cache = A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D)
    dev = to_device(q, cache)
    qt, qv = rows_in(rng, 12, Hq, D, torch.bfloat16)
    batch = q.KvBatch(i32(table), i32(lens), 12, 3, i32(cu_of(ns)))
    need = q.moe_attn_decode_workspace_bytes(dev, batch, Hq)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(qt, 9.0), torch.full((12, Hq), 9.0, device="cuda")
    q.moe_attn_decode(dev, batch, qt, out, ws[:need], 0.09, lse)
    assert torch.all(ws[need:] == 0x5A)
    assert torch.all(out[3:9] == 9.0) and torch.all(lse[3:9] == 9.0)
    for b, rows in ((0, slice(0, 3)), (1, slice(9, 12))):
        K, V, _ = cache.read(table[b], 0, lens[b])
        seen = np.arange(lens[b])[None] <= (lens[b] - ns[b] + np.arange(3))[:, None]
        ref, rl, mag, smag = A.attention(qv[rows], K, V, seen, 0.09)
        check_attention(out[rows], lse[rows], ref, rl, *attention_bounds(torch.bfloat16, D, V, ref, mag, smag, lens[b]), f"sequence {b}")


def test_decode_is_repeatable_and_needs_no_clean_workspace(q):
    rng = np.random.default_rng(34)
    Hk, D, page, lens = 2, 128, 64, [5000, 300, 4097]
    table, n_pages = page_table(rng, lens, page)
    dev = to_device(q, A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D))
    qt, _ = rows_in(rng, 3, 16, D, torch.bfloat16)
    batch = _batch(q, table, lens, [1, 1, 1], uniform=True)
    got = []
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((q.moe_attn_decode_workspace_bytes(dev, batch, 16),), fill, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(qt), torch.empty((3, 16), device="cuda")
        q.moe_attn_decode(dev, batch, qt, out, ws, 0.1, lse)
        got.append((out, lse))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_cache_offsets_past_32_bits(q):
    """A 4.5 GB cache whose sequence lies in its last pages: append, read, decode."""
    rng = np.random.default_rng(35)
    Hk, D, page, L = 4, 128, 64, 90
    per = q.moe_kv_code_bytes(1, page, Hk, D)
    n_pages = (9 << 29) // per
    dev = q.KvCache(None, None, page, Hk, D, n_pages)
    table = np.array([[n_pages - 1, n_pages - 2]])
    kt, _ = rows_in(rng, L, Hk, D, torch.bfloat16)
    vt, _ = rows_in(rng, L, Hk, D, torch.bfloat16)
    batch = _batch(q, table, [L], [L])
    q.moe_kv_append(dev, batch, kt, vt)
    k, v = torch.empty_like(kt), torch.empty_like(vt)
    q.moe_kv_read(dev, batch, k, v)
    ref = A.Cache(np.zeros((2, Hk, page // 16, 2, 16 * D), np.uint8), np.zeros((2, Hk, page // 16, 2)), page, Hk, D)
    ref.append([1, 0], 0, f64(kt), f64(vt))
    K, V, _ = ref.read([1, 0], 0, L)
    assert np.array_equal(f64(k), K) and np.array_equal(f64(v), V)
    assert np.array_equal(dev.codes[-2 * per:].cpu().numpy().reshape(ref.codes.shape)[0][:, 0], ref.codes[0][:, 0])
    qt, qv = rows_in(rng, 1, 8, D, torch.bfloat16)
    step = _batch(q, table, [L], [1])
    ws = torch.empty(q.moe_attn_decode_workspace_bytes(dev, step, 8), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(qt), torch.empty((1, 8), device="cuda")
    q.moe_attn_decode(dev, step, qt, out, ws, 0.1, lse)
    o, rl, mag, smag = A.attention(qv, K, V, np.ones((1, L), bool), 0.1)
    check_attention(out, lse, o, rl, *attention_bounds(torch.bfloat16, D, V, o, mag, smag, L), "last pages")


# ---------------------------------------------------------------------------
# prefill


def _prefill(q, ns, ms, Hq, Hk, D, dt, causal, rng, what, sigma=1.0, spoil=None, extra=0, pad=0, max_q=None):
    dt = DT[dt]
    Tq, Tk = sum(ns) + extra, sum(ms) + extra
    qt, qv = rows_in(rng, Tq, Hq, D, dt, pad=pad, sigma=sigma)
    kt, kv = rows_in(rng, Tk, Hk, D, dt, pad=2 * pad)
    vt, vv = rows_in(rng, Tk, Hk, D, dt)
    if spoil:
        spoil(kt, vt)
        kv, vv = f64(kt), f64(vt)
    out = torch.full((Tq, Hq * D + pad), 9.0, dtype=dt, device="cuda")[:, :Hq * D].unflatten(1, (Hq, D))
    lse = torch.full((Tq, Hq), 9.0, device="cuda")
    cuq, cuk = cu_of(ns), cu_of(ms)
    mq = max(max(ns), 1) if max_q is None else max_q
    ws = torch.full((q.moe_attn_prefill_workspace_bytes(Tq, len(ns), mq, Tk, Hq, Hk, D),), 0xFF, dtype=torch.uint8, device="cuda")
    scale = D ** -0.5
    q.moe_attn_prefill(qt, kt, vt, i32(cuq), i32(cuk), mq, out, ws, scale, causal, lse)
    torch.cuda.synchronize()
    assert torch.all(out[cuq[-1]:] == 9.0) and torch.all(lse[cuq[-1]:] == 9.0)
    for b, (n, m) in enumerate(zip(ns, ms)):
        r, k = slice(cuq[b], cuq[b + 1]), slice(cuk[b], cuk[b + 1])
        seen = np.arange(m)[None] <= (m - n + np.arange(n))[:, None] if causal else np.ones((n, m), bool)
        ref, rl, mag, smag = A.attention(qv[r], kv[k], vv[k], seen, scale)
        tol, tl = attention_bounds(dt, D, vv[k], ref, mag, smag, m)
        check_attention(out[r], lse[r], ref, rl, tol, tl, f"{what}, sequence {b}")
    return out, lse


PREFILL = [  # query rows, key rows, query heads, key heads
    ([1], [1], 1, 1),
    ([5, 1, 33], [5, 1, 33], 4, 2),
    ([64, 65, 0, 127], [64, 65, 7, 127], 2, 2),
    ([10, 4, 3], [200, 0, 1], 6, 2),                   # a chunk's end, no keys, more rows than keys
    ([130], [321], 8, 1),
    ([1, 1, 1, 1], [1, 63, 64, 65], 3, 1),
    # enough heads to fill the card with row tiles of 128
    ([5, 64, 127], [5, 64, 127], 64, 64),
    ([3, 40, 100], [65, 300, 99], 128, 32),
    ([129, 0, 9], [7, 3, 0], 48, 24),                  # (24 key heads on 8 XCDs)
    ([60, 65], [60, 400], 99, 33),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill(q, case, D, causal, dt):
    ns, ms, Hq, Hk = PREFILL[case]
    rng = np.random.default_rng(300 + case)
    _prefill(q, ns, ms, Hq, Hk, D, dt, causal, rng, f"case {case}", sigma=2.0, extra=3, pad=16)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D,heads", [(64, 1), (128, 1), (128, 64), (64, 64), (256, 1), (256, 64)])
def test_prefill_special_values(q, D, heads, dt):
    """Infinities and NaN in keys and values reach the rows that see them, and no row before their token."""
    def spoil(k, v):
        v[60, 0, 3], v[61, 0, 9], v[90, 0, 33], v[100, 0, 0] = float("inf"), -float("inf"), float("nan"), float("nan")
        v[100, 0, 63], v[129, 0, 5] = float("inf"), float("inf")
        k[110, 0, 7] = float("nan")
        v[139, 0, :] = float("nan")                    # the last key of the first sequence
    rng = np.random.default_rng(36)
    _prefill(q, [140, 30], [140, 30], 2 * heads, heads, D, dt, True, rng, "special values", spoil=spoil)


def test_prefill_longer(q):
    rng = np.random.default_rng(37)
    _prefill(q, [300, 700], [300, 1100], 4, 1, 128, "bf16", True, rng, "longer", sigma=3.0)
    _prefill(q, [513], [513], 4, 4, 64, "fp16", True, rng, "longer, narrow", sigma=3.0, max_q=2000)
    _prefill(q, [300, 517], [300, 800], 32, 32, 128, "bf16", True, rng, "longer, many heads", sigma=3.0)
    _prefill(q, [200, 333], [700, 800], 48, 16, 64, "fp16", False, rng, "longer, many heads, all keys", sigma=3.0)


def test_prefill_few_rows_many_keys(q):
    rng = np.random.default_rng(38)
    _prefill(q, [3, 20], [2500, 3333], 4, 2, 128, "bf16", True, rng, "few rows", sigma=2.0)
    _prefill(q, [9], [2049], 2, 2, 64, "fp16", False, rng, "few rows, narrow")
    _prefill(q, [1, 2, 0], [700, 5, 40], 2, 1, 256, "bf16", True, rng, "few rows, wide heads")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_parts(q, D, dt):
    """Keys cut into parts: of unequal contexts, so that a sequence's last parts have no tiles, with empty sequences."""
    rng = np.random.default_rng(49)
    Hq, Hk, ns, ms = 4, 1, [5, 0, 40], [3500, 700, 90]
    assert q.moe_attn_prefill_workspace_bytes(45, 3, 40, sum(ms), Hq, Hk, D) > 256
    _prefill(q, ns, ms, Hq, Hk, D, dt, True, rng, "parts", sigma=2.0)
    _prefill(q, ns, ms, Hq, Hk, D, dt, False, rng, "parts, all keys", sigma=2.0, pad=8)


@pytest.mark.parametrize("Tk", [300, 6000])
def test_prefill_in_a_graph(q, Tk):
    """A captured call, whole and cut into parts, replayed with other rows and another cut into sequences: the eager
    call's bits."""
    rng = np.random.default_rng(50)
    Hq, Hk, D, Tq, dt = 4, 2, 128, 60, torch.bfloat16
    xs = [[rows_in(rng, n, h, D, dt)[0] for n, h in ((Tq, Hq), (Tk, Hk), (Tk, Hk))] for _ in range(4)]
    cus = [(i32([0, a, Tq]), i32([0, b, Tk])) for a, b in ((30, Tk // 2), (1, Tk - 7), (59, 3), (20, Tk // 3))]
    ws = [torch.empty(q.moe_attn_prefill_workspace_bytes(Tq, 2, Tq, Tk, Hq, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert (ws[0].numel() > 256) == (Tk == 6000)
    x, cu = [t.clone() for t in xs[0]], [t.clone() for t in cus[0]]
    out, lse = torch.zeros((Tq, Hq, D), dtype=dt, device="cuda"), torch.zeros((Tq, Hq), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q.moe_attn_prefill(*x, *cu, Tq, out, ws[0], 0.09, True, lse)
    for i in range(12):
        for dst, src in zip(x + cu, xs[i % 4] + list(cus[i % 4])):
            dst.copy_(src)
        graph.replay()
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        q.moe_attn_prefill(*xs[i % 4], *cus[i % 4], Tq, o, ws[1], 0.09, True, l)
        if i % 3 == 2:
            torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("n_keys", [70, 9000])
def test_prefill_more_rows_than_max_q(q, n_keys):
    """A sequence with more rows than max_q says, whole and cut into parts: the first max_q are right, the others untouched."""
    rng = np.random.default_rng(46)
    Hk, D, Hq, ns, ms, most = 2, 128, 4, [41, 7], [n_keys, 50], 9
    qt, qv = rows_in(rng, sum(ns), Hq, D, torch.bfloat16)
    kt, kv = rows_in(rng, sum(ms), Hk, D, torch.bfloat16)
    vt, vv = rows_in(rng, sum(ms), Hk, D, torch.bfloat16)
    need = q.moe_attn_prefill_workspace_bytes(sum(ns), 2, most, sum(ms), Hq, Hk, D)
    assert (need > 256) == (n_keys == 9000)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(qt, 9.0), torch.full((sum(ns), Hq), 9.0, device="cuda")
    q.moe_attn_prefill(qt, kt, vt, i32(cu_of(ns)), i32(cu_of(ms)), most, out, ws[:need], 0.09, True, lse)
    assert torch.all(ws[need:] == 0x5A)
    assert torch.all(out[most:41] == 9.0) and torch.all(lse[most:41] == 9.0)
    for b, (rows, keys) in enumerate(((slice(0, most), slice(0, n_keys)), (slice(41, 48), slice(n_keys, n_keys + 50)))):
        seen = np.arange(ms[b])[None] <= (ms[b] - ns[b] + np.arange(rows.stop - rows.start))[:, None]
        K, V = kv[keys], vv[keys]
        ref, rl, mag, smag = A.attention(qv[rows], K, V, seen, 0.09)
        check_attention(out[rows], lse[rows], ref, rl, *attention_bounds(torch.bfloat16, D, V, ref, mag, smag, ms[b]), f"sequence {b}")


def test_prefill_no_keys_at_all(q):
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.ones_like(x), torch.zeros((3, 2), device="cuda")
    ws = torch.empty(q.moe_attn_prefill_workspace_bytes(3, 1, 3, 0, 2, 2, 64), dtype=torch.uint8, device="cuda")
    q.moe_attn_prefill(x, k, k, i32([0, 3]), i32([0, 0]), 3, out, ws, 0.1, True, lse)
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


# ---------------------------------------------------------------------------
# together


def test_prompt_in_chunks_then_steps(q):
    """A user's run: two prompts go in as odd chunks (turn, append, read the context back, attend), then single-token
    and draft steps over the cache.  Each call's output is checked on what the calls before it left."""
    rng = np.random.default_rng(40)
    Hq, Hk, D, page, dt = 8, 2, 128, 64, torch.bfloat16
    table, n_pages = page_table(rng, [400, 300], page)
    codes, scales = random_cache(rng, n_pages, page, Hk, D, garbage=True)
    dev = to_device(q, A.Cache(codes, scales, page, Hk, D))
    rope = q.Rope(torch.from_numpy(q.moe_rope_freqs(D, rule="parts", factor=4, trained=256)).cuda(), D, False, 1.1)
    scale = D ** -0.5
    lens = np.array([0, 0])
    for ns in ([200, 77], [100, 130]):
        lens = lens + ns
        T = sum(ns)
        qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hk, D))).to(dt).cuda()
        qs, ks, vs = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        q.moe_kv_append(dev, _batch(q, table, lens, ns), ks, vs, rope, qs, qs)
        Tk = int(sum(lens))
        k, v = (torch.empty((Tk, Hk, D), dtype=dt, device="cuda") for _ in range(2))
        q.moe_kv_read(dev, _batch(q, table, lens, list(lens)), k, v)
        out, lse = torch.empty((T, Hq, D), dtype=dt, device="cuda"), torch.empty((T, Hq), device="cuda")
        ws = torch.empty(q.moe_attn_prefill_workspace_bytes(T, 2, max(ns), Tk, Hq, Hk, D), dtype=torch.uint8, device="cuda")
        q.moe_attn_prefill(qs, k, v, i32(cu_of(ns)), i32(cu_of(lens)), max(ns), out, ws, scale, True, lse)
        # the same rows through the decode call, which reads the codes: the two agree with the oracle
        out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
        step = _batch(q, table, lens, ns)
        ws2 = torch.empty(q.moe_attn_decode_workspace_bytes(dev, step, Hq), dtype=torch.uint8, device="cuda")
        q.moe_attn_decode(dev, step, qs, out2, ws2, scale, lse2)
        cu, cuk = cu_of(ns), cu_of(lens)
        for b in (0, 1):
            r, kk = slice(cu[b], cu[b + 1]), slice(cuk[b], cuk[b + 1])
            seen = np.arange(lens[b])[None] <= (lens[b] - ns[b] + np.arange(ns[b]))[:, None]
            ref, rl, mag, smag = A.attention(f64(qs[r]), f64(k[kk]), f64(v[kk]), seen, scale)
            bounds = attention_bounds(dt, D, f64(v[kk]), ref, mag, smag, lens[b])
            check_attention(out[r], lse[r], ref, rl, *bounds, f"chunk, sequence {b}")
            check_attention(out2[r], lse2[r], ref, rl, *bounds, f"chunk over the cache, sequence {b}")
    for ns in ([1, 1], [3, 1], [1, 2]):
        lens = lens + ns
        T = sum(ns)
        qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hk, D))).to(dt).cuda()
        step = _batch(q, table, lens, ns)
        q_out = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        q.moe_kv_append(dev, step, qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], rope, qkv[:, :Hq], q_out)
        cache = A.Cache(dev.codes.cpu().numpy(), f64(dev.scales), page, Hk, D)
        out, lse = torch.empty_like(q_out), torch.empty((T, Hq), device="cuda")
        ws = torch.empty(q.moe_attn_decode_workspace_bytes(dev, step, Hq), dtype=torch.uint8, device="cuda")
        q.moe_attn_decode(dev, step, q_out, out, ws, scale, lse)
        cu = cu_of(ns)
        for b in (0, 1):
            r = slice(cu[b], cu[b + 1])
            K, V, _ = cache.read(table[b], 0, int(lens[b]))
            seen = np.arange(lens[b])[None] <= (lens[b] - ns[b] + np.arange(ns[b]))[:, None]
            ref, rl, mag, smag = A.attention(f64(q_out[r]), K, V, seen, scale)
            check_attention(out[r], lse[r], ref, rl, *attention_bounds(dt, D, V, ref, mag, smag, lens[b]), f"step, sequence {b}")


@pytest.mark.parametrize("width", [None, 200])
def test_steps_in_a_graph_on_a_side_stream(q, width):
    """A captured step (append, attend) replayed with lengths and rows that the program moves on between replays equals
    the eager steps, to the bit; contexts whole, and cut into ranges (a wide page table)."""
    rng = np.random.default_rng(41)
    Hq, Hk, D, page, dt, steps = 8, 2, 128, 16, torch.bfloat16, 20
    table, n_pages = page_table(rng, [60, 90], page, width=width)
    codes, scales = random_cache(rng, n_pages, page, Hk, D)
    rows = torch.from_numpy(rng.standard_normal((steps, 2, Hq + 2 * Hk, D))).to(dt).cuda()
    rope = q.Rope(torch.from_numpy(q.moe_rope_freqs(D)).cuda(), D)
    got = {}
    for mode in ("eager", "graph"):
        dev = to_device(q, A.Cache(codes, scales, page, Hk, D))
        lens = i32([40, 70])
        batch = q.KvBatch(i32(table), lens, 2)
        x = torch.zeros_like(rows[0])
        q_out, out, lse = (torch.zeros((2, Hq, D), dtype=dt, device="cuda"), torch.zeros((2, Hq, D), dtype=dt, device="cuda"),
                           torch.zeros((2, Hq), device="cuda"))
        ws = torch.empty(q.moe_attn_decode_workspace_bytes(dev, batch, Hq), dtype=torch.uint8, device="cuda")

        def step():
            q.moe_kv_append(dev, batch, x[:, Hq:Hq + Hk], x[:, Hq + Hk:], rope, x[:, :Hq], q_out)
            q.moe_attn_decode(dev, batch, q_out, out, ws, 0.09, lse)

        graph = None
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        outs = []
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for i in range(steps):
                x.copy_(rows[i])
                lens += 1
                graph.replay() if graph else step()
                outs.append((out.clone(), lse.clone()))
                if i % 5 == 4:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        got[mode] = (outs, dev.codes.clone(), dev.scales.clone())
    for (a, la), (b, lb) in zip(got["eager"][0], got["graph"][0]):
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert torch.equal(got["eager"][1], got["graph"][1]) and torch.equal(got["eager"][2], got["graph"][2])


@pytest.mark.parametrize("width", [None, 400])
def test_layer_steps_in_a_graph(q, width):
    """Attention and the routed experts as one captured step: rows in, turned and appended, attended to, and through
    the layer that takes the heads' outputs as its input.  Replays equal the eager steps to the bit, and the experts'
    output is the oracle's for the attention's."""
    import synth
    from layer_fixture import device_layer, oracle_layer, rel_err
    wl = synth.WORKLOADS["tiny"]
    layer = device_layer(wl)
    rng = np.random.default_rng(47)
    H, E, k = wl.hidden, wl.n_experts, wl.top_k
    Hq, Hk, D, page, dt, steps, B = 4, 2, H // 4, 16, torch.bfloat16, 8, 3
    table, _ = page_table(rng, [40, 60, 300], page, width=width)
    n_pages = int(table.max()) + 1
    codes, scales = random_cache(rng, n_pages, page, Hk, D)
    rows = torch.from_numpy(rng.standard_normal((steps, B, Hq + 2 * Hk, D)) * 3).to(dt).cuda()
    rope = q.Rope(torch.from_numpy(q.moe_rope_freqs(D)).cuda(), D)
    got = {}
    for mode in ("eager", "graph"):
        dev = to_device(q, A.Cache(codes, scales, page, Hk, D))
        lens = i32([20, 47, 280])
        batch = q.KvBatch(i32(table), lens, B)
        x = torch.zeros_like(rows[0])
        q_out, out = torch.zeros((B, Hq, D), dtype=dt, device="cuda"), torch.zeros((B, Hq, D), dtype=dt, device="cuda")
        idx, w = torch.zeros((B, k), dtype=torch.int32, device="cuda"), torch.zeros((B, k), device="cuda")
        y = torch.zeros((B, H), device="cuda")
        ws = torch.empty(q.moe_attn_decode_workspace_bytes(dev, batch, Hq), dtype=torch.uint8, device="cuda")
        lws = torch.empty(q.moe_layer_decode_workspace_bytes(layer.w, B, k), dtype=torch.uint8, device="cuda")

        def step():
            q.moe_kv_append(dev, batch, x[:, Hq:Hq + Hk], x[:, Hq + Hk:], rope, x[:, :Hq], q_out)
            q.moe_attn_decode(dev, batch, q_out, out, ws, 0.3)
            q.moe_layer_decode(layer.w, layer.router, None, out.view(B, H), B, k, idx, w, y, lws)

        graph = None
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for i in range(steps):
            x.copy_(rows[i])
            lens += 1
            graph.replay() if graph else step()
            outs.append([t.clone() for t in (out, idx, w, y)])
        torch.cuda.synchronize()
        got[mode] = outs
    for e, g in zip(got["eager"], got["graph"]):
        assert all(torch.equal(a, b) for a, b in zip(e, g))
    for e in got["eager"][::3]:
        ref, ref_idx, _ = oracle_layer(wl, f64(e[0]).reshape(B, H))
        assert np.array_equal(e[1].cpu().numpy(), ref_idx)
        assert rel_err(e[3].cpu().numpy(), ref).max() <= 2e-3


def test_two_streams_at_once(q):
    """Two sequences attended to on two streams, each call with a workspace of its own: as one after the other."""
    rng = np.random.default_rng(42)
    Hk, D, page = 2, 128, 64
    table, n_pages = page_table(rng, [9000, 7000], page)
    dev = to_device(q, A.Cache(*random_cache(rng, n_pages, page, Hk, D), page, Hk, D))
    xs = [rows_in(rng, 1, 16, D, torch.bfloat16)[0] for _ in range(2)]
    batches = [_batch(q, table[b:b + 1], [[9000, 7000][b]], [1]) for b in range(2)]
    ws = [torch.empty(q.moe_attn_decode_workspace_bytes(dev, s, 16), dtype=torch.uint8, device="cuda") for s in batches]
    want = [torch.empty_like(x) for x in xs]
    for b in range(2):
        q.moe_attn_decode(dev, batches[b], xs[b], want[b], ws[b], 0.1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(x) for _ in range(10)] for x in xs]
    for i in range(10):
        for b in range(2):
            q.moe_attn_decode(dev, batches[b], xs[b], outs[b][i], ws[b], 0.1, stream=streams[b])
    torch.cuda.synchronize()
    for b in range(2):
        for o in outs[b]:
            assert torch.equal(o, want[b])


def test_binding_refusals(q):
    """Each argument the binding looks at, wrong in each way: refused with its name, and nothing written."""
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = x[:, :2]
    dev = q.KvCache(torch.zeros(4 * 2 * 16 * 2 * 64, dtype=torch.uint8, device="cuda"), torch.zeros(16, device="cuda"), 16, 2, 64)
    batch = q.KvBatch(i32([[0], [1]]), i32([1, 1]), 2)
    ws = torch.empty(q.moe_attn_decode_workspace_bytes(dev, batch, 4), dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, 7.0)
    turned = x.transpose(1, 2).contiguous().transpose(1, 2)                        # heads not back to back
    wrong = {"too few rows": x[:1], "another type": x.float(), "not its q's type": x.half(), "on the host": x.cpu(), "no tensor": 3,
             "two dimensions": x[0], "heads apart": turned, "another dimension": x[:, :, :32]}
    f32 = torch.zeros((2, 4), device="cuda")
    cu = i32([0, 1, 2])

    def refuses(call, name, what):
        with pytest.raises((ValueError, q.QmoeError), match=name if isinstance(name, str) else None):
            call()
            pytest.fail(f"{what} was not refused")

    for what, bad in wrong.items():
        b2 = bad if not isinstance(bad, torch.Tensor) or bad.dim() != 3 else bad[:, :2]
        if what != "not its q's type":
            refuses(lambda: q.moe_attn_decode(dev, batch, bad, out, ws, 0.1), "q", f"decode q {what}")
            refuses(lambda: q.moe_kv_append(dev, batch, b2, kv), "k", f"append k {what}")
            refuses(lambda: q.moe_kv_read(dev, batch, b2, out[:, :2]), "k_out", f"read k_out {what}")
        if what not in ("too few rows", "another dimension", "not its q's type"):
            refuses(lambda: q.moe_attn_prefill(bad, kv, kv, cu, cu, 1, out, ws, 0.1), "q", f"prefill q {what}")
        if what != "too few rows":
            refuses(lambda: q.moe_attn_prefill(x, b2, kv, cu, cu, 1, out, ws, 0.1), "k|v", f"prefill k {what}")
        refuses(lambda: q.moe_attn_decode(dev, batch, x, bad, ws, 0.1), "out", f"decode out {what}")
        refuses(lambda: q.moe_attn_prefill(x, kv, kv, cu, cu, 1, bad, ws, 0.1), "out", f"prefill out {what}")
        refuses(lambda: q.moe_attn_prefill(x, kv, b2, cu, cu, 1, out, ws, 0.1), "v", f"prefill v {what}")
        refuses(lambda: q.moe_kv_append(dev, batch, kv, b2), "v", f"append v {what}")
        refuses(lambda: q.moe_kv_append(dev, batch, kv, kv, None, bad, out), "q|q_out", f"append q {what}")
        refuses(lambda: q.moe_kv_append(dev, batch, kv, kv, None, x, bad), "q_out", f"append q_out {what}")
        refuses(lambda: q.moe_kv_append(dev, batch, kv, kv, None, None, None, b2), "k_out", f"append k_out {what}")
        refuses(lambda: q.moe_kv_read(dev, batch, out[:, :2], b2), "v_out", f"read v_out {what}")
    for what, bad in {"too small": f32[0], "another type": f32.half(), "on the host": f32.cpu(), "strided": torch.zeros((4, 4), device="cuda")[:, :2]}.items():
        refuses(lambda: q.moe_attn_decode(dev, batch, x, out, ws, 0.1, bad), "lse", f"decode lse {what}")
        refuses(lambda: q.moe_attn_prefill(x, kv, kv, cu, cu, 1, out, ws, 0.1, True, bad), "lse", f"prefill lse {what}")
    for bad in (None, f32, ws.cpu(), ws[::2]):
        refuses(lambda: q.moe_attn_decode(dev, batch, x, out, bad, 0.1), "ws", "decode ws")
        refuses(lambda: q.moe_attn_prefill(x, kv, kv, cu, cu, 1, out, bad, 0.1), "ws", "prefill ws")
    for bad in (None, cu.long(), cu.cpu(), cu[:1]):
        refuses(lambda: q.moe_attn_prefill(x, kv, kv, bad, cu, 1, out, ws, 0.1), "cu_q", "cu_q")
        refuses(lambda: q.moe_attn_prefill(x, kv, kv, cu, bad, 1, out, ws, 0.1), "cu_k", "cu_k")
    for call in (lambda: q.moe_attn_decode(dev, batch, x, out, ws[:100], 0.1),       # too small a workspace
                 lambda: q.moe_attn_decode(dev, batch, x, out, ws, float("nan")),
                 lambda: q.moe_attn_decode(dev, batch, x[:, :3], out[:, :3], ws, 0.1),   # heads that do not divide
                 lambda: q.moe_attn_prefill(x, kv, kv, cu, cu, 0, out, ws, 0.1),
                 lambda: q.moe_attn_prefill(x, kv, kv, cu, cu, 1 << 40, out, ws, 0.1),
                 lambda: q.moe_attn_prefill(x[:, :0], kv, kv, cu, cu, 1, out[:, :0], ws, 0.1),
                 lambda: q.moe_kv_append(dev, batch, kv, kv, None, x, None),         # q without q_out
                 lambda: q.moe_kv_append(dev, batch, kv, kv, None, None, out),
                 lambda: q.moe_kv_append(dev, batch, x, x),                          # another number of heads
                 lambda: q.moe_kv_read(dev, batch, kv, None),
                 lambda: q.KvBatch(i32([[0, 1], [1, 2]]).t(), i32([1, 1]), 2),
                 lambda: q.KvBatch(i32([[0], [1]]), i32([1, 1]), 2, None, i32([0, 1, 2])),
                 lambda: q.KvCache(torch.zeros(100, dtype=torch.uint8, device="cuda"), None, 16, 2, 64)):
        refuses(call, None, "call")
    for call in (lambda: q.moe_attn_decode(dev, batch, x, out, ws, "0.1"), lambda: q.moe_attn_prefill(x, kv, kv, cu, cu, 1.5, out, ws, 0.1)):
        with pytest.raises(TypeError):
            call()
    torch.cuda.synchronize()
    assert torch.all(out == 7.0) and not dev.codes.any() and not dev.scales.any()
    # and what is not wrong: more rows than the step has, one head of a row with odd strides
    q.moe_attn_decode(dev, batch, torch.cat([x, x]), torch.cat([out, out]), ws, 1, f32)
    one = q.KvCache(dev.codes, dev.scales, 16, 1, 64)
    y = torch.zeros((2, 24, 64), dtype=torch.bfloat16, device="cuda")[:, 5:6]
    q.moe_kv_append(one, batch, y, y, None, y, y)
    torch.cuda.synchronize()
