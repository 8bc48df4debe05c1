"""Plain forms of a serving step over the 4-bit cache, for the tests: pages and places,
block summaries, block selection, attention over lists of positions. numpy and Python
integers on the host, written from the definitions in xp.h, no code of the package."""
from __future__ import annotations

import numpy as np

import attn_ref as ref


def ends(counts):
    return np.concatenate([[0], np.cumsum(np.asarray(counts, dtype=np.int64))]).astype(np.int32)


# ---------------------------------------------------------- pages and places
def plan(lens, want, table, free, count, rows, page, n_pages):
    """One sequence after the other: (cu, start, lens_out, seq, pos, slot); table and the stack's height change."""
    batch, cols = table.shape
    height = min(max(count, 0), n_pages)
    cu, lens_out, seq, pos, slot = [0], [], [], [], []
    asked = [0, 0]
    for b in range(batch):
        n, w = int(lens[b]), int(want[b])
        asks = w > 0 and n >= 0 and n + w <= cols * page
        if asks:
            first, end = -(-n // page), -(-(n + w) // page)
            asked = [asked[0] + w, asked[1] + end - first]
        if asks and asked[0] <= rows and asked[1] <= height:
            for c in range(first, end):
                table[b, c] = free[height - 1 - (asked[1] - (end - first)) - (c - first)]
            for p in range(n, n + w):
                seq.append(b)
                pos.append(p)
            cu.append(cu[-1] + w)
            lens_out.append(n + w)
            taken = asked[1]
        else:
            if asks:                              # nobody behind it is served
                asked = [1 << 62, 1 << 62]
            cu.append(cu[-1])
            lens_out.append(n)
    taken = sum(-(-lens_out[b] // page) - -(-int(lens[b]) // page) for b in range(batch) if lens_out[b] != lens[b])
    for b, p in zip(seq, pos):
        t = int(table[b, p // page])
        slot.append(t * page + p % page if 0 <= t < n_pages else -1)
    fill = [-1] * (rows - len(seq))
    return (np.array(cu), np.array(lens), np.array(lens_out), np.array(seq + fill), np.array(pos + fill),
            np.array(slot + fill, dtype=np.int64), height - taken)


def release(lens, keep, table, free, count, page, n_pages):
    height = min(max(count, 0), n_pages)
    for b in reversed(range(table.shape[0])):
        n, k = min(int(lens[b]), table.shape[1] * page), max(int(keep[b]), 0)
        if n <= k:
            continue
        for c in reversed(range(-(-k // page), -(-n // page))):
            if 0 <= table[b, c] < n_pages:
                if height < n_pages:
                    free[height] = table[b, c]
                height += 1
            table[b, c] = -1
    return min(height, n_pages)


# ------------------------------------------------------------- cached values
def tile_values(cache, tile, which):
    """A tile's 64 rows [64][dim] and their scale bytes [64][ng], from its bytes."""
    at = [cache.at(0, 0, p, which) for p in range(64)]
    codes = np.stack([(tile[c] >> (4 * odd)) & 15 for c, odd, _ in at])
    byte = np.stack([tile[s] for _, _, s in at])
    return codes, byte


def cached(cache, table_row, head, n, which):
    """As Cache.rows, a tile at a time: values [n][dim] of positions 0 .. n-1 and which of them the cache has."""
    out, there = np.zeros((n, cache.dim)), np.zeros(n, dtype=bool)
    for p in range(0, n, 64):
        page = int(table_row[p // cache.page])
        if 0 <= page < cache.pages:
            codes, byte = tile_values(cache, cache.b[page, head, (p % cache.page) // 64], which)
            m = min(64, n - p)
            out[p:p + m] = ref.values(codes, byte)[:m]
            there[p:p + m] = True
    return out, there


# ------------------------------------------------------------ block summaries
UNITS = [0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12]            # halves


def scale_units(b):
    """An E4M3 byte in units of 2^-9, 0 for a NaN."""
    e, m = (b >> 3) & 15, b & 7
    v = 0 if (b & 127) == 127 else (m if e == 0 else (8 + m) << (e - 1))
    return -v if b >= 128 else v


SCALE_UNITS = np.array([scale_units(b) for b in range(256)], dtype=np.int64)


def summary(codes, byte):
    """The signed bytes and k of a block of 64 keys."""
    v = np.array(UNITS, dtype=np.int64)[codes] * np.repeat(SCALE_UNITS[byte], 32, axis=-1)
    total = [int(x) for x in v.sum(0)]
    k = 0
    while max(abs(x) for x in total) > 127 << k:
        k += 1

    def nearest(x):
        q, r = divmod(x, 1 << k)
        return q + (1 if 2 * r > 1 << k or (2 * r == 1 << k and q % 2) else 0)
    return np.array([nearest(x) for x in total], dtype=np.int64), k


def entry_of(cache, page, head, tile):
    return (page * cache.kv + head) * (cache.page // 64) + tile


def summarise(cache, out, cu, start, table):
    """Into `out` (the buffer's bytes) the blocks that the rows complete."""
    entries = cache.pages * cache.kv * (cache.page // 64)
    for b in range(len(start)):
        for r in range(cu[b], cu[b + 1]):
            p = int(start[b]) + int(r - cu[b])
            if p < 0 or p >= table.shape[1] * cache.page or p % 64 != 63:
                continue
            page = int(table[b, p // cache.page])
            if not 0 <= page < cache.pages:
                continue
            for h in range(cache.kv):
                t = (p % cache.page) // 64
                code, k = summary(*tile_values(cache, cache.b[page, h, t], "k"))
                e = entry_of(cache, page, h, t)
                out[e * cache.dim:(e + 1) * cache.dim] = code.astype(np.int8).view(np.uint8)
                out[entries * cache.dim + e] = k


# ------------------------------------------------------------------ selection
def steps_of(x):
    """A head's q in whole steps of 2^e and e; zeros and None where it is zero or not finite."""
    top = np.max(np.abs(x))
    if not np.isfinite(x).all() or top == 0:
        return np.zeros(len(x), dtype=np.int64), None
    e = int(np.floor(np.log2(top))) - 8
    while top > 127 * 2.0 ** e:
        e += 1
    assert top > 127 * 2.0 ** (e - 1)
    return np.rint(x * 2.0 ** -e).astype(np.int64), e


def scores(q, codes, ks):
    """q [group][dim], codes [blocks][dim], ks [blocks]: the blocks' scores, exact in float64."""
    heads = [steps_of(x) for x in q]
    known = [e for _, e in heads if e is not None]
    top = max(known) if known else 0
    s = [(codes @ x) * (2.0 ** max(e - top, -64) if e is not None else 0.0) for x, e in heads]
    return np.max(s, axis=0) * 2.0 ** ks.astype(np.float64)


def select(score, there, n, keep, sinks, recent):
    """The blocks of [0, n) that are listed."""
    if n <= keep:
        return list(range(n))
    order = sorted(range(sinks, n - recent), key=lambda j: (not there[j], -score[j] if there[j] else 0.0, j))
    return sorted(list(range(sinks)) + order[:keep - sinks - recent] + list(range(n - recent, n)))
