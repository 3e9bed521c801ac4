"""Plain fp64 oracle of the attention calls (include/qmoe_attn.h): rotary
positions, the paged 8-bit cache (layout, scale rule, growth), attention.
Numpy only; shares no code with the kernels.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16

# the 8-bit format: 4 exponent bits (bias 7), 3 of mantissa, no infinities
_MAG = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)])
_MAG[127] = np.nan


def e4m3_decode(codes):
    c = np.asarray(codes, np.uint8)
    return np.where(c >> 7, -1.0, 1.0) * _MAG[c & 127]


def e4m3_encode(x):
    """Nearest code, ties to the even mantissa; |x| <= 448 or not finite (code 0x7F or 0xFF)."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    assert a.size == 0 or a.max() <= 464, "outside the format"
    hi = np.clip(np.searchsorted(_MAG[:127], a), 1, 126)
    lo = hi - 1
    dl, dh = a - _MAG[lo], _MAG[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = np.where(np.isfinite(x), code, 127)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def least_scale(amax):
    """Least power of two s >= 2^-64 with amax <= 448 s."""
    if amax == 0:
        return 2.0 ** -64
    k = math.floor(math.log2(amax / 448.0)) - 1
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** max(k, -64)


def rotate(x, pos, freqs, interleaved=False, scale=1.0):
    """x [n, heads, D] at positions pos [n]: the first 2 len(freqs) columns turned."""
    y = np.array(x, np.float64)
    r = len(freqs)
    for i, f in enumerate(freqs):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        t = (np.asarray(pos, np.float64) * f)[:, None]
        y[..., u] = scale * (x[..., u] * np.cos(t) - x[..., v] * np.sin(t))
        y[..., v] = scale * (x[..., u] * np.sin(t) + x[..., v] * np.cos(t))
    return y


def k_offset(n, d):
    """Byte of token n, column d among a block's K codes."""
    c = 16 * (d % 32 // 8) + n
    return 1024 * (d // 64) + 16 * c + 8 * (d % 64 // 32) + d % 8


def v_offset(n, d):
    return 1024 * (d // 64) + 16 * (16 * (n // 4) + d % 16) + 4 * (d % 64 // 16) + n % 4


class Cache:
    """The cache of include/qmoe_attn.h as arrays; codes [pages, heads, blocks, 2, 16 D], scales [pages, heads, blocks, 2]."""

    def __init__(self, codes, scales, page, heads, dim):
        self.page, self.heads, self.dim = page, heads, dim
        self.codes = np.array(codes, np.uint8).reshape(-1, heads, page // BLOCK, 2, BLOCK * dim)
        self.scales = np.array(scales, np.float64).reshape(-1, heads, page // BLOCK, 2)
        n, d = np.meshgrid(np.arange(BLOCK), np.arange(dim), indexing="ij")
        self.at = (k_offset(n, d), v_offset(n, d))

    def block(self, table, pos):
        """(page, block) that holds position pos, or None."""
        page = int(table[pos // self.page])
        return None if page < 0 or page >= len(self.codes) else (page, pos % self.page // BLOCK)

    def append(self, table, first, k, v):
        """k, v [n, heads, D] (fp64) at positions first..first+n-1 (those below 0 left out)."""
        n = len(k)
        lo = max(first, 0)
        for b0 in range(lo // BLOCK * BLOCK, first + n, BLOCK):
            at = self.block(table, b0)
            if at is None:
                continue
            s, e = max(lo - b0, 0), min(first + n - b0, BLOCK)
            for part, x in ((0, k), (1, v)):
                for h in range(self.heads):
                    new = x[b0 + s - first:b0 + e - first, h]
                    fin = np.abs(new[np.isfinite(new)])
                    now = least_scale(fin.max() if fin.size else 0.0)
                    bits = self.codes[at[0], h, at[1], part]
                    if s > 0:
                        was = self.scales[at[0], h, at[1], part]
                        now = max(now, was)
                        if now > was:
                            w = self.at[part][:s]
                            bits[w] = e4m3_encode(e4m3_decode(bits[w]) * (was / now))
                    bits[self.at[part][s:e]] = e4m3_encode(new / now)
                    self.scales[at[0], h, at[1], part] = now

    def read(self, table, lo, hi):
        """K, V [hi-lo, heads, D] of positions lo..hi-1, and which of them a page holds; zeros for the others."""
        K = np.zeros((hi - lo, self.heads, self.dim))
        V = np.zeros_like(K)
        there = np.zeros(hi - lo, bool)
        for p in range(max(lo, 0), hi):
            at = self.block(table, p)
            if at is None:
                continue
            there[p - lo] = True
            for part, to in ((0, K), (1, V)):
                c = self.codes[at[0], :, at[1], part][:, self.at[part][p % BLOCK]]
                to[p - lo] = e4m3_decode(c) * self.scales[at[0], :, at[1], part][:, None]
        return K, V, there


def attention(q, k, v, seen, scale):
    """q [n, Hq, D], k and v [m, Hk, D], seen [n, m]: out [n, Hq, D], lse [n, Hq]; rows that see nothing give 0 and
    -inf.  A key a row does not see plays no part in it, whatever it holds.  Two sums that bound rounding errors:
    sum p |v| like out, and the largest scale * sum |q| |k| of a row like lse."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, mag, smag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    lse = np.full((n, Hq), -np.inf)
    for i in range(n):
        js = np.nonzero(seen[i])[0]
        if not len(js):
            continue
        for h in range(Hq):
            with np.errstate(invalid="ignore", over="ignore"):
                s = k[js, h // g] @ q[i, h] * scale
                smag[i, h] = (np.abs(k[js, h // g]) @ np.abs(q[i, h]) * scale).max()
                m = s.max()
                if m == -np.inf:
                    continue
                p = np.exp(s - m)
                out[i, h] = p @ v[js, h // g] / p.sum()
                mag[i, h] = p @ np.abs(v[js, h // g]) / p.sum()
                lse[i, h] = m + np.log(p.sum())
    return out, lse, mag, smag
