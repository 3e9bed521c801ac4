"""Plain CPU forms, in 64 bits, of the calls around attention and the experts (norm, 4-bit products, pages of a cache).
Shares no code with the library; for tests."""
import numpy as np

from .qmoe_oracle import f16

BLOCK = 16


# ---------------------------------------------------------------------------
# Norm.

def add(x, residual, to_type):
    """x + residual in 32 bits (both exact in them), rounded to the residual's type by to_type."""
    return to_type((np.asarray(x, np.float32) + np.asarray(residual, np.float32)).astype(np.float64))


def rms_norm(h, weight, eps):
    """Vectors along the last axis."""
    h = np.asarray(h, np.float64)
    with np.errstate(all="ignore"):
        return h / np.sqrt((h * h).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * weight


def codes8(y, group):
    """int8 codes and fp32 scales [.., groups] of vectors along the last axis."""
    n = y.shape[-1]
    group = group or n
    codes = np.zeros(y.shape, np.int8)
    scales = np.zeros(y.shape[:-1] + (-(-n // group),), np.float32)
    with np.errstate(all="ignore"):
        for g, at in enumerate(range(0, n, group)):
            part = y[..., at:at + group]
            m = np.abs(part).max(-1).astype(np.float32)
            s = (m.astype(np.float64) / 127).astype(np.float32)
            fine = np.isfinite(m)
            use = fine & (s > 0)
            q = np.rint(part / np.where(use, s, 1).astype(np.float64)[..., None])
            codes[..., at:at + group] = np.where(use[..., None], np.clip(np.nan_to_num(q), -127, 127), 0)
            scales[..., g] = np.where(fine, s, np.nan)
    return codes, scales


# ---------------------------------------------------------------------------
# 4-bit products.

def quantize4(w, group, with_zeros):
    w = np.asarray(w, np.float64)
    n, k = w.shape
    gn = -(-k // group)
    q, s, z = np.zeros((n, k), np.uint8), np.zeros((n, gn)), np.full((n, gn), 8, np.uint8)
    for g in range(gn):
        x = w[:, g * group:(g + 1) * group]
        lo, hi = np.minimum(x.min(1), 0), np.maximum(x.max(1), 0)
        s[:, g] = f16((hi - lo) / 15 if with_zeros else (np.maximum(-lo, hi) + 0.0) / 7)
        d = np.where(s[:, g] > 0, s[:, g], 1)
        if with_zeros:
            z[:, g] = np.where(s[:, g] > 0, np.clip(np.floor(-lo / d + 0.5), 0, 15), 8)
        c = np.clip(np.floor(x / d[:, None] + 0.5) + z[:, g, None], 0, 15)
        q[:, g * group:(g + 1) * group] = np.where(s[:, g, None] > 0, c, 8)
    return q, s, z


def weights4(q, s, z, group):
    k = q.shape[1]
    up = lambda a: np.repeat(np.asarray(a, np.float64), group, 1)[:, :k]  # noqa: E731
    return (q.astype(np.float64) - up(z)) * up(s)


def pack4(q, s, z, group):
    """Bytes of the tiles, value by value; z None: without zero points."""
    n, k = q.shape
    gt, gn = 128 // group, s.shape[1]
    rt, kc = -(-n // 16), -(-k // 128)
    size = 1024 + 32 * gt + (16 * gt if z is not None else 0)
    out = np.zeros((rt * kc, size), np.uint8)
    half = np.asarray(s, np.float16).view(np.uint16)
    for row in range(n):
        for col in range(k):
            t, r, c = out[row // 16 * kc + col // 128], row % 16, col % 128
            word, g, j = c // 32, c % 32 // 8, c % 8
            bit = 4 * (j // 2) + 16 * (j % 2)
            t[16 * (16 * g + r) + 4 * word + bit // 8] |= (int(q[row, col]) ^ 8) << (bit % 8)
        for g in range(gn):
            t, r, i = out[row // 16 * kc + g // gt], row % 16, g % gt
            at = 1024 + 2 * gt * r + 2 * i
            t[at], t[at + 1] = half[row, g] & 255, half[row, g] >> 8
            if z is not None:
                t[1024 + 32 * gt + gt * r + i] = (int(z[row, g]) - 8) & 255
    return out.reshape(-1)


def product(x, w, bias=None):
    """x w^T (+ bias) and the sums of the terms' sizes."""
    with np.errstate(all="ignore"):
        y = np.asarray(x, np.float64) @ w.T
        mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, mag


# ---------------------------------------------------------------------------
# Pages.

class Pages:
    """A pool, the rows of a page table, and what the pages hold (any array whose first axis is the page, or layer and
    page, and whose block axis is the one that `blocks` cuts)."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.page = [list(r) for r in table], list(lens), list(refs), page
        self.copies = []                   # (from, to, blocks)

    def length(self, v):
        return min(max(int(v), 0), len(self.table[0]) * self.page)

    def held(self, v):
        return -(-self.length(v) // self.page)

    def _release(self, p):
        if 0 <= p < len(self.refs):
            self.refs[p] -= 1

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def resize(self, new):
        rows = [b for b, n in enumerate(new) if n >= 0]
        for b in rows:
            for i in range(self.held(new[b]), self.held(self.lens[b])):
                self._release(self.table[b][i])
                self.table[b][i] = -1
        free, used, missing = self._free(), 0, 0
        for b in rows:
            have, want = self.held(self.lens[b]), self.held(new[b])
            if want > have:
                used += want - have
                if used > len(free):
                    missing += want - have
                    continue
                for i in range(have, want):
                    p = free[used - want + i]
                    self.table[b][i], self.refs[p] = p, 1
            self.lens[b] = self.length(new[b])
        return missing

    def fork(self, origin):
        before = [self.length(x) for x in self.lens]
        tables, refs = [list(r) for r in self.table], list(self.refs)
        free, used, missing = self._free(), 0, 0
        inside = lambda p: 0 <= p < len(refs)  # noqa: E731
        for b, a in enumerate(origin):
            if not 0 <= a < len(before) or before[a] == 0:
                continue
            full, rest = divmod(before[a], self.page)
            last = tables[a][full] if rest else -1
            if a == b:
                if not rest or not inside(last) or refs[last] <= 1:
                    continue
            elif before[b]:
                continue
            if rest:
                used += 1
                if used > len(free):
                    missing += 1
                    continue
            if a != b:
                for i in range(full):
                    p = tables[a][i]
                    self.table[b][i] = p
                    if inside(p):
                        self.refs[p] += 1
                self.lens[b] = before[a]
            else:
                self.refs[last] -= 1
            if rest:
                p = free[used - 1]
                self.table[b][full], self.refs[p] = p, self.refs[p] + 1
                if inside(last):
                    self.copies.append((last, p, -(-rest // BLOCK)))
        return missing

    def compact(self):
        n = sum(r != 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        moving = [p for p in range(n, len(self.refs)) if self.refs[p] != 0]
        to = dict(zip(moving, holes))
        for b, x in enumerate(self.lens):
            for i in range(self.held(x)):
                self.table[b][i] = to.get(self.table[b][i], self.table[b][i])
        for p, t in to.items():
            self.refs[t], self.refs[p] = self.refs[p], 0
            self.copies.append((p, t, self.page // BLOCK))
        return n
