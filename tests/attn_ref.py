"""Plain float64 forms of the 4-bit cache and of attention, for the tests: numpy on
the host, written from the definitions in xp.h, no code of the package."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=np.float64)


def _e4m3_table():
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = np.nan if (b & 127) == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) / 8 * 2.0 ** (e - 7))
        t[b] = -v if b >= 128 else v
    return t


E4M3 = _e4m3_table()
SCALES = E4M3[:127]                      # 0 .. 448, rising


def quantise(x):
    """x [..., dim] float64 -> codes [..., dim] (0..15) and scale bytes [..., dim / 32]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(g).all(-1)
    a = np.where(np.isfinite(g), np.abs(g), 0.0)
    byte = np.minimum(np.searchsorted(6.0 * SCALES, a.max(-1), side="left"), 126)
    s = SCALES[byte][..., None]
    # e2m1 magnitudes of even code win a tie: compare with the seven midpoints
    code = np.zeros(g.shape, dtype=np.uint8)
    for n, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += ((a > mid * s) if n % 2 == 0 else (a >= mid * s)).astype(np.uint8)
    code = np.where((s > 0) & ~bad[..., None], code, 0).astype(np.uint8)
    code = code | (np.signbit(g).astype(np.uint8) << 3)
    return code.reshape(x.shape), np.where(bad, 127, byte).astype(np.uint8)


def values(codes, byte):
    return E2M1[codes] * np.repeat(E4M3[byte], 32, axis=-1)


class Cache:
    """A cache as its bytes [pages][kv_heads][tiles][tile bytes]."""

    def __init__(self, kv_heads, dim, page, pages, fill=None, rng=None):
        self.kv, self.dim, self.page, self.pages, self.ng = kv_heads, dim, page, pages, dim // 32
        shape = (pages, kv_heads, page // 64, self.ng * 2176)
        self.b = np.zeros(shape, dtype=np.uint8) if rng is None else rng.integers(0, 256, shape, dtype=np.uint8)
        if fill is not None:
            self.b[...] = fill

    def at(self, page, head, off, which):
        """Byte offsets (codes [dim], whose low or high nibble [dim], scales [ng]) inside a tile."""
        pos, d, g, ng = off % 64, np.arange(self.dim), np.arange(self.ng), self.ng
        if which == "k":
            return ((d // 32) * 1024 + pos * 16 + (d % 32) // 2, d % 2,
                    ng * 1024 + g * 64 + (pos % 16) * 4 + pos // 16)
        return (ng * 1088 + (d // 16) * 512 + pos * 8 + (d % 16) // 2, d % 2,
                ng * 2112 + g * 64 + (pos // 4 % 4) * 16 + (pos // 16) * 4 + pos % 4)

    def put(self, page, head, off, which, codes, byte):
        tile = self.b[page, head, off // 64]
        c, odd, s = self.at(page, head, off, which)
        lo, hi = codes[0::2], codes[1::2]
        tile[c[0::2]] = lo | (hi << 4)
        tile[s] = byte

    def get(self, page, head, off, which):
        tile = self.b[page, head, off // 64]
        c, odd, s = self.at(page, head, off, which)
        return (tile[c] >> (4 * odd)) & 15, tile[s]

    def rows(self, table_row, head, n, which):
        """Values [n][dim] of positions 0 .. n-1 and which of them the cache has."""
        out, there = np.zeros((n, self.dim)), np.zeros(n, dtype=bool)
        for p in range(n):
            page = int(table_row[p // self.page])
            if 0 <= page < self.pages:
                there[p] = True
                out[p] = values(*self.get(page, head, p % self.page, which))
        return out, there


def append(cache, k, v, cu, start, table):
    for b in range(len(start)):
        for r in range(cu[b], cu[b + 1]):
            p = int(start[b]) + r - cu[b]
            if p < 0 or p >= table.shape[1] * cache.page or not 0 <= table[b, p // cache.page] < cache.pages:
                continue
            for h in range(cache.kv):
                for which, x in (("k", k), ("v", v)):
                    cache.put(int(table[b, p // cache.page]), h, p % cache.page, which, *quantise(x[r, h]))


def attend(q, k, v, at, scale, window=0, there=None, out_step=0.0, p_step=0.0):
    """q [rows][dim] at positions `at` over k, v [n][dim]: out, p, and a bound on a kernel's error.

    The bound: an output's own rounding, half a step `out_step` of its value; each
    probability's rounding, `p_step`; scores and sums in fp32: (dim + n) steps of 2^-24 on
    what is summed in absolute value (a score of magnitude S moves its exponential by S times
    its relative error), all times the sum of p |v|. The exponential, its argument's rounding
    and the reciprocal add a few 2^-22."""
    n = len(k)
    j = np.arange(n)
    see = j[None, :] <= np.asarray(at)[:, None]
    if window:
        see &= j[None, :] > np.asarray(at)[:, None] - window
    if there is not None:
        see &= there[None, :]
    with np.errstate(all="ignore"):
        s = (q @ k.T) * scale
        mag = scale * (np.abs(q) @ np.abs(k).T)
        s = np.where(see, s, -np.inf)
        top = np.max(s, axis=1, keepdims=True) if n else np.full((len(q), 1), -np.inf)
        p = np.exp(s - np.where(np.isneginf(top), 0.0, top))
        p = np.where(see, p, 0.0)
        tot = p.sum(1, keepdims=True)
        p = np.where(tot == 0, 0.0, p / np.where(tot == 0, 1.0, tot))
        # what a row does not see takes no part, NaN and infinities included
        out = np.zeros((len(q), v.shape[1]))
        wide = np.zeros_like(out)
        for i in range(len(q)):
            out[i] = p[i, see[i]] @ v[see[i]]
            wide[i] = p[i, see[i]] @ np.abs(v[see[i]])
        big = np.where(see, mag, 0.0).max(1, keepdims=True) if n else np.zeros((len(q), 1))
        rel = p_step + (v.shape[1] + n) * 2.0 ** -24 * (1.0 + big) + 2.0 ** -20
        return out, p, out_step * np.abs(out) + rel * wide + 1e-30, rel


def evict_list(w, n, keep, sinks, recent):
    """Positions kept of n with weights w (numpy fp32)."""
    if n <= keep:
        return np.arange(n)
    lo, hi = sinks, n - recent
    x = np.asarray(w[lo:hi], dtype=np.float64) + 0.0
    # NaN below every number; equal weights by lower position
    order = sorted(range(hi - lo), key=lambda i: ((1, 0.0) if np.isnan(x[i]) else (0, -x[i]), i))
    mid = np.array(sorted(order[:keep - sinks - recent]), dtype=np.int64) + lo
    return np.concatenate([np.arange(lo), mid, np.arange(hi, n)]).astype(np.int64)
