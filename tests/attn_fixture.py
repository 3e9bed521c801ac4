"""Shared by the attention tests: caches, steps, tolerances."""
import numpy as np

import torch

from oracle import attn_oracle as A

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def subnormal_half(dt):
    """Half the distance of the type's subnormal numbers."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def cu_of(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rows_in(rng, n, heads, dim, dt, pad=0, sigma=1.0):
    """A row tensor of n rows (rows `pad` elements further apart than they are long) and its values."""
    x = torch.from_numpy(rng.standard_normal((n, heads, dim)) * sigma).to(dt)
    buf = torch.full((n, heads * dim + pad), float("nan"), dtype=dt, device="cuda")
    view = buf[:, :heads * dim].unflatten(1, (heads, dim))
    view.copy_(x)
    return view, f64(x)


def page_table(rng, lens, page, width=None, spare=1, order=None):
    """Pages of sequences of these lengths, in random order; entries behind a sequence's pages name no page."""
    need = [-(-l // page) for l in lens]
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages) if order is None else order
    width = max(max(need), 1) if width is None else width
    t = np.full((len(lens), width), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, n_pages


def random_cache(rng, n_pages, page, heads, dim, sigma=1.0, garbage=False):
    """Codes and scales of normally distributed values (numpy); garbage: not-a-number codes and scales everywhere."""
    shape = (n_pages, heads, page // A.BLOCK, 2)
    if garbage:
        return np.full(shape + (A.BLOCK * dim,), 0x7F, np.uint8), np.full(shape, np.nan)
    codes = A.e4m3_encode(np.clip(rng.standard_normal(shape + (A.BLOCK * dim,)) * 112, -448, 448))
    return codes, sigma * 2.0 ** rng.integers(-8, -5, shape)


def spoil_tails(cache, table, lens):
    """Not-a-number codes in every slot behind a sequence's last token, and in pages no sequence has."""
    used = set()
    for b, n in enumerate(lens):
        for p in range(-(-n // cache.page)):
            used.add(int(table[b, p]))
        nb = -(-n // A.BLOCK) * A.BLOCK
        for pos in range(n, nb):
            at = cache.block(table[b], pos)
            for part in (0, 1):
                cache.codes[at[0], :, at[1], part][:, cache.at[part][pos % A.BLOCK]] = 0x7F
        for b0 in range(nb, -(-n // cache.page) * cache.page, A.BLOCK):
            at = cache.block(table[b], b0)
            cache.codes[at[0], :, at[1]] = 0xFF
            cache.scales[at[0], :, at[1]] = np.nan
    for p in set(range(len(cache.codes))) - used:
        cache.codes[p] = 0x7F
        cache.scales[p] = np.nan


def to_device(q, cache):
    codes = torch.from_numpy(cache.codes.reshape(-1)).cuda()
    scales = torch.from_numpy(cache.scales.astype(np.float32).reshape(-1)).cuda()
    return q.KvCache(codes, scales, cache.page, cache.heads, cache.dim)


def in_type(x, dt):
    """fp64 values rounded to the row type."""
    return torch.from_numpy(x).to(dt).to(torch.float64).numpy()


def rounded(x, dt):
    """fp64 values rounded once to the row type (torch rounds them to 32 bits on the way)."""
    bits, least = (8, -125) if dt == torch.bfloat16 else (11, -13)
    quantum = np.ldexp(1.0, np.maximum(np.frexp(x)[1], least) - bits)
    return np.rint(x / quantum) * quantum


def attention_bounds(dt, dim, v, out, mag, smag, n_keys):
    """How far outputs and log sums may be from the oracle's, from the arithmetic alone.

    Scores: products of 16-bit values are exact in 32 bits, so a score is off by at most dim + 2 roundings of its
    partial sums (none larger than smag / scale), one for scale * log2(e), one for the product with it, one for the
    subtraction of the maximum: e_s in all, a relative e_s of exp.  exp2 itself is good to 2^-21.  The
    weights are rounded to the row type (half a step; below the smallest normal number half a subnormal step of
    the largest weight, 1), the sums over keys are 32-bit (n_keys roundings at most, and the joins'), the
    output is rounded once more."""
    smag = np.where(np.isfinite(smag), smag, 0)
    e_s = (dim + 5) * 2.0 ** -24 * smag + 2.0 ** -21
    rel = half_step(dt) + 2 * e_s + (n_keys + 16) * 2.0 ** -23
    vmax = np.abs(v[np.isfinite(v)]).max() if np.isfinite(v).any() else 0.0
    tol = rel[..., None] * mag * (1 + 2 ** -6) + half_step(dt) * np.abs(out) + subnormal_half(dt) * (n_keys * vmax + 1)
    return tol, e_s + (n_keys + 16) * 2.0 ** -23 + 2.0 ** -20


def check_attention(got, lse, ref, ref_lse, tol, tol_lse, what):
    got, lse = f64(got), f64(lse)
    for name, g, r, t in (("out", got, ref, tol), ("lse", lse, ref_lse, tol_lse + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0)))):
        fine = np.isfinite(r)
        assert np.array_equal(np.isnan(g), np.isnan(r)), f"{what}: {name}: not a number elsewhere than the oracle"
        assert np.array_equal(g[~fine & ~np.isnan(r)], r[~fine & ~np.isnan(r)]), f"{what}: {name}: infinities differ"
        d = np.abs(g - np.where(fine, r, 0))[fine]
        lim = np.broadcast_to(t, r.shape)[fine]
        worst = (d / lim).max() if d.size else 0.0
        assert worst <= 1, f"{what}: {name} is {worst:.2f} times its bound off (largest error {d.max():.3e})"
