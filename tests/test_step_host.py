"""Host side of a serving step's entry points (no GPU): sizes, refusals before any launch,
and the tests' own references against independent checks."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref
import step_ref as step

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)
BF16, F16, F32 = 0, 1, 2
INF, NAN = float("inf"), float("nan")
BAD_DIMS = [(0, 64, 64, 4), (1025, 64, 64, 4), (2, 96, 64, 4), (2, 512, 64, 4), (2, 64, 0, 4), (2, 64, 96, 4), (2, 64, 64, 0)]


def kd(kv=2, dim=64, page=64, pages=4):
    return ctypes.byref(xp.kv_dims(kv, dim, page, pages))


def at(n):
    """An address of its own for every array, far from the others."""
    return ctypes.c_void_p((n + 1) << 40)


def call(name, base, kw):
    a = dict(base, **kw)
    return getattr(xp.lib(), name)(*[a[k] for k in base], None)


PLAN = dict(g=kd(), batch=3, cols=2, rows=8, lens=at(0), want=at(1), table=at(2), free=at(3), count=at(4), cu=at(5), start=at(6),
            out=at(7), seq=at(8), pos=at(9), slot=at(10))
RELEASE = dict(g=kd(), batch=3, cols=2, lens=at(0), keep=at(1), table=at(2), free=at(3), count=at(4))
BLOCKS = dict(g=kd(), batch=1, cols=1, rows=64, cu=at(0), start=at(1), table=at(2), cache=at(3), blocks=at(4))
SELECT = dict(g=kd(), heads=4, batch=1, cols=4, rows=3, ty=BF16, q=at(0), qs=256, cu=at(1), start=at(2), table=at(3), blocks=at(4),
              keep=3, sinks=1, recent=1, sel=at(5))
SPARSE = dict(g=kd(), heads=4, batch=1, cols=4, rows=3, keep=3, ty=BF16, q=at(0), qs=256, scale=1.0, cache=at(1), table=at(2),
              cu=at(3), start=at(4), sel=at(5), out=at(6), os=256, ws=at(7), bytes=1 << 40)
CHUNK = dict(g=kd(), heads=4, batch=1, cols=4, rows=3, max_len=256, ty=BF16, q=at(0), qs=256, scale=1.0, window=0, cache=at(1),
             table=at(2), cu=at(3), start=at(4), out=at(5), os=256, ws=at(6), bytes=1 << 40)
CALLS = {"xp_kv_plan": PLAN, "xp_kv_release": RELEASE, "xp_kv_blocks": BLOCKS, "xp_attn_select": SELECT, "xp_attn_sparse": SPARSE,
         "xp_attn_chunk": CHUNK}
POINTERS = {n: [k for k, v in base.items() if isinstance(v, ctypes.c_void_p)] for n, base in CALLS.items()}


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_dims_and_null_pointers_are_refused(name):
    for d in BAD_DIMS:
        assert call(name, CALLS[name], dict(g=kd(*d))) == xp.XP_ERR_SHAPE, d
    assert call(name, CALLS[name], dict(g=None)) == xp.XP_ERR_NULL
    for key in POINTERS[name]:
        assert call(name, CALLS[name], {key: None}) == xp.XP_ERR_NULL, key
        assert call(name, CALLS[name], {key: ctypes.c_void_p(0x1003)}) == xp.XP_ERR_SHAPE, key
    for kw in (dict(batch=-1), dict(batch=65536), dict(cols=0), dict(cols=1 << 26)):
        assert call(name, CALLS[name], kw) == xp.XP_ERR_SHAPE, kw
    none = {k: None for k in POINTERS[name]}
    assert call(name, CALLS[name], dict(none, batch=0)) == xp.XP_OK
    if name not in ("xp_kv_plan", "xp_kv_release"):
        assert call(name, CALLS[name], dict(none, rows=0)) == xp.XP_OK


@pytest.mark.parametrize("name", list(CALLS))
def test_shapes_out_of_range_are_refused(name):
    bad = {"xp_kv_plan": [dict(rows=-1), dict(rows=(1 << 24) + 1)], "xp_kv_release": [],
           "xp_kv_blocks": [dict(rows=-1), dict(rows=2 ** 31 - 1), dict(g=kd(kv=1024), rows=64 * ((1 << 13) - 1) + 1)],
           "xp_attn_select": [dict(rows=-1), dict(rows=1 << 21), dict(heads=0), dict(heads=3), dict(heads=65536), dict(ty=F32), dict(ty=5),
                              dict(qs=255), dict(qs=250), dict(qs=260), dict(keep=0, sinks=0), dict(keep=1), dict(sinks=-1),
                              dict(recent=0), dict(sinks=2, recent=2), dict(keep=16385), dict(cols=16385), dict(q=ctypes.c_void_p(0x1008)),
                              dict(blocks=ctypes.c_void_p(0x1008))]}
    many = [dict(rows=-1), dict(heads=0), dict(heads=3), dict(heads=65536), dict(ty=F32), dict(ty=-1), dict(qs=248), dict(qs=260),
            dict(os=252), dict(os=258), dict(scale=0.0), dict(scale=-1.0), dict(scale=INF), dict(scale=NAN),
            dict(q=ctypes.c_void_p(0x1008)), dict(out=ctypes.c_void_p(0x1004)), dict(cache=ctypes.c_void_p(0x1008)),
            dict(ws=ctypes.c_void_p(0x1008))]
    bad["xp_attn_sparse"] = many + [dict(keep=0), dict(keep=(1 << 24) + 1), dict(rows=1 << 23)]
    bad["xp_attn_chunk"] = many + [dict(window=-1), dict(max_len=-1), dict(rows=2 ** 31 - 1, heads=2),
                                   dict(rows=1 << 28, heads=2 * 8, qs=1024, os=1024)]
    for kw in bad[name]:
        assert call(name, CALLS[name], kw) == xp.XP_ERR_SHAPE, kw


def test_overlaps_are_refused():
    for base, name, written in ((PLAN, "xp_kv_plan", ("table", "count", "cu", "start", "out", "seq", "pos", "slot")),
                                (RELEASE, "xp_kv_release", ("table", "free", "count"))):
        for w in written:
            for other in POINTERS[name]:
                if w == other or (w, other) == ("out", "lens"):
                    continue
                assert call(name, base, {other: base[w]}) == xp.XP_ERR_SHAPE, (w, other)
    # the free pages' room behind the stack's top counts as well
    assert call("xp_kv_plan", PLAN, dict(count=ctypes.c_void_p(PLAN["free"].value + 12))) == xp.XP_ERR_SHAPE
    assert call("xp_kv_blocks", BLOCKS, dict(blocks=ctypes.c_void_p(BLOCKS["cache"].value + 4096))) == xp.XP_ERR_SHAPE
    assert call("xp_attn_select", SELECT, dict(sel=SELECT["q"])) == xp.XP_ERR_SHAPE
    for name in ("xp_attn_sparse", "xp_attn_chunk"):
        q = CALLS[name]["q"].value
        assert call(name, CALLS[name], dict(out=ctypes.c_void_p(q + 8))) == xp.XP_ERR_SHAPE
        assert call(name, CALLS[name], dict(out=ctypes.c_void_p(q), os=264)) == xp.XP_ERR_SHAPE


def test_workspaces():
    d = xp.kv_dims(2, 128, 64, 4)
    need = xp.xp_attn_chunk_workspace_bytes(d, 8, 40, 2, 9000)
    assert need > 16
    assert xp.xp_attn_chunk_workspace_bytes(d, 8, 40, 2, 100) == 16          # nothing is cut
    assert call("xp_attn_chunk", CHUNK, dict(g=ctypes.byref(d), heads=8, rows=40, batch=2, max_len=9000, qs=1024, os=1024,
                                             bytes=need - 1)) == xp.XP_ERR_WORKSPACE
    need = xp.xp_attn_sparse_workspace_bytes(d, 8, 1, 400)
    assert need > 16 and xp.xp_attn_sparse_workspace_bytes(d, 8, 1000, 400) == 16
    assert call("xp_attn_sparse", SPARSE, dict(g=ctypes.byref(d), heads=8, rows=1, keep=400, qs=1024, os=1024,
                                               bytes=need - 1)) == xp.XP_ERR_WORKSPACE
    for bad in BAD_DIMS:
        g = xp.kv_dims(*bad)
        assert xp.xp_kv_blocks_bytes(g) == 0
        assert xp.xp_attn_chunk_workspace_bytes(g, 4, 1, 1, 64) == 0 and xp.xp_attn_sparse_workspace_bytes(g, 4, 1, 4) == 0
    assert xp.lib().xp_kv_blocks_bytes(None) == 0
    for kv, dim, page, pages in ((8, 128, 256, 10), (1, 64, 64, 1), (3, 256, 192, 7)):
        assert xp.xp_kv_blocks_bytes(xp.kv_dims(kv, dim, page, pages)) == pages * page // 64 * kv * (dim + 1)


# ------------------------------------------------------------------ references
def test_plan_by_hand():
    """Page 64, a table of three columns: lengths 60, 64, 10, 0, 5 ask for 5, 1, 0, 200, 1."""
    table = np.full((5, 3), -1)
    table[0, 0], table[1, 0], table[2, 0], table[4, 0] = 0, 1, 2, 3
    free = np.array([9, 8, 7, 6, -1])
    cu, start, lens, seq, pos, slot, height = step.plan([60, 64, 10, 0, 5], [5, 1, 0, 200, 1], table, free, 4, 8, 64, 10)
    assert cu.tolist() == [0, 5, 6, 6, 6, 7] and lens.tolist() == [65, 65, 10, 0, 6]      # 200 do not fit the table
    assert table.tolist() == [[0, 6, -1], [1, 7, -1], [2, -1, -1], [-1, -1, -1], [3, -1, -1]] and height == 2
    assert seq.tolist() == [0, 0, 0, 0, 0, 1, 4, -1] and pos.tolist() == [60, 61, 62, 63, 64, 64, 5, -1]
    assert slot.tolist() == [60, 61, 62, 63, 6 * 64, 7 * 64, 3 * 64 + 5, -1]
    assert step.release(lens, [60, 64, 10, 0, 5], table, free, height, 64, 10) == 4
    assert free.tolist() == [9, 8, 7, 6, -1] and table[:, 1].tolist() == [-1] * 5
    # the first that does not fit ends it, though a later one would
    table = np.full((3, 3), -1)
    cu, _, _, _, _, _, height = step.plan([0, 0, 0], [3, 4, 1], table, np.arange(9), 9, 6, 64, 9)
    assert cu.tolist() == [0, 3, 3, 3] and height == 8
    cu, _, _, _, _, _, height = step.plan([0, 0, 0], [3, 70, 1], table, np.arange(9), 2, 600, 64, 9)
    assert cu.tolist() == [0, 3, 3, 3] and height == 1


def test_summary_against_exact_fractions():
    rng = np.random.default_rng(1)
    for _ in range(20):
        codes, byte = rng.integers(0, 16, (64, 64)), rng.integers(0, 256, (64, 2))
        total = []
        for d in range(64):
            s = Fraction(0)
            for p in range(64):
                b = int(byte[p, d // 32])
                if (b & 127) != 127:
                    s += Fraction(float(ref.E2M1[codes[p, d]])) * Fraction(float(ref.E4M3[b]))
            total.append(s * 1024)
        assert all(t.denominator == 1 and abs(t) < 1 << 28 for t in total)
        got, k = step.summary(codes, byte)
        assert max(abs(t) for t in total) <= 127 << k and (k == 0 or max(abs(t) for t in total) > 127 << (k - 1))
        assert got.tolist() == [round(t / (1 << k)) for t in total]          # Python rounds fractions to even
        assert np.abs(got).max() <= 127


def test_steps_and_scores():
    q = np.array([0.5, -0.25, 1.0, 0.003])
    got, e = step.steps_of(q)
    assert e == -6 and got.tolist() == [32, -16, 64, 0]
    assert step.steps_of(np.array([127.0 / 128]))[1] == -7 and step.steps_of(np.array([127.5 / 128]))[1] == -6
    assert step.steps_of(np.zeros(3))[1] is None and step.steps_of(np.array([1.0, np.inf]))[1] is None
    codes, ks = np.array([[1, 2, 3, 4], [5, 0, -7, 0]]), np.array([3, 1])
    s = step.scores(np.array([q, -2 * q]), codes, ks)
    # the second head's steps are twice the first's: 32 - 32 + 192 = 192 and -288 -> * 2^-1, 0
    assert s.tolist() == [max(192 * 0.5, -192.0) * 8, max((160 - 448) * 0.5, 288.0) * 2]


def test_select_by_hand():
    s = np.array([9, 1, 5, 5, 7, 5, 0, 0], dtype=np.float64)
    there = np.ones(8, dtype=bool)
    assert step.select(s, there, 8, 8, 1, 1) == list(range(8)) and step.select(s, there, 0, 3, 1, 1) == []
    assert step.select(s, there, 8, 5, 1, 1) == [0, 2, 3, 4, 7]             # 7, then the lower ones of the fives
    assert step.select(s, there, 8, 2, 1, 1) == [0, 7]
    there[4] = False
    assert step.select(s, there, 8, 5, 1, 1) == [0, 2, 3, 5, 7]
    there[:] = False
    assert step.select(s, there, 8, 4, 1, 2) == [0, 1, 6, 7]


def test_cached_is_the_caches_rows():
    rng = np.random.default_rng(3)
    c = ref.Cache(2, 64, 128, 5, rng=rng)
    c.b[..., :] %= 127
    table = np.array([4, -1, 2, 5, 0])
    for which in "kv":
        for n in (0, 1, 63, 64, 65, 300, 640):
            a, b = c.rows(table, 1, n, which), step.cached(c, table, 1, n, which)
            np.testing.assert_array_equal(a[0], b[0])
            np.testing.assert_array_equal(a[1], b[1])


def test_columns_of_pages_and_launch_limits():
    """Both sides of the launches' limits: what is just below passes the checks and is refused for its small workspace."""
    g = kd(kv=1, dim=64)
    a = dict(g=g, heads=1, qs=64, os=64, bytes=0)
    assert call("xp_attn_sparse", SPARSE, dict(a, rows=(1 << 24) - 1)) == xp.XP_ERR_WORKSPACE
    assert call("xp_attn_sparse", SPARSE, dict(a, rows=1 << 24)) == xp.XP_ERR_SHAPE
    rows = 256 * ((1 << 23) - 600)                                            # wide blocks, and the cut pieces' workgroups
    assert call("xp_attn_chunk", CHUNK, dict(a, rows=rows)) == xp.XP_ERR_WORKSPACE
    assert call("xp_attn_chunk", CHUNK, dict(a, rows=256 * (1 << 23) - 300)) == xp.XP_ERR_SHAPE
