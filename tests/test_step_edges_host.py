"""Host side of a serving step's entry points at their edges (no GPU): an empty batch, outputs
over inputs, workspaces."""
import ctypes
import itertools

import pytest

from fp4_routed_expert_xp_amd import xp

from test_step_host import BLOCKS, CHUNK, PLAN, SELECT, SPARSE, at, call


# ---------------------------------------------------------------- empty batch
def test_plan_without_sequences_checks_what_it_writes():
    """Arrays that are there are held to the same rules as with sequences; those that are not are left out."""
    none = {k: None for k, v in PLAN.items() if isinstance(v, ctypes.c_void_p)}
    assert call("xp_kv_plan", PLAN, dict(none, batch=0)) == xp.XP_OK
    for key in ("cu", "seq", "pos", "slot"):
        assert call("xp_kv_plan", PLAN, dict(none, batch=0, **{key: ctypes.c_void_p(0x1002)})) == xp.XP_ERR_SHAPE, key
    assert call("xp_kv_plan", PLAN, dict(none, batch=0, slot=ctypes.c_void_p(0x1004))) == xp.XP_ERR_SHAPE
    for a, b in (("cu", "seq"), ("seq", "pos"), ("pos", "slot"), ("cu", "slot")):
        assert call("xp_kv_plan", PLAN, dict(none, batch=0, **{a: at(1), b: at(1)})) == xp.XP_ERR_SHAPE, (a, b)
    assert call("xp_kv_plan", PLAN, dict(none, batch=0, seq=at(1), pos=ctypes.c_void_p(at(1).value + 28))) == xp.XP_ERR_SHAPE
    # without rows the maps are empty, wherever they lie
    assert call("xp_kv_plan", PLAN, dict(none, batch=0, rows=0, seq=at(1), pos=at(1), slot=at(1))) == xp.XP_OK


# ------------------------------------------------------------- outputs over inputs
def test_chosen_blocks_are_not_written_over():
    """out [3][4][64] of two bytes in rows of os elements, sel [3][2][3] int32: 72 bytes."""
    base = SPARSE["out"].value
    for where, os_, bad in ((0, 256, True), (-68, 256, True), (-72, 256, False), (3 * 512 - 4, 256, True), (3 * 512, 256, False),
                            # rows 2,048 bytes apart leave room for it, but not everywhere
                            (512, 1024, False), (2048 - 72, 1024, False), (2048 - 68, 1024, True), (2048 + 508, 1024, True)):
        kw = dict(out=ctypes.c_void_p(base), os=os_, sel=ctypes.c_void_p(base + where), bytes=0)
        assert call("xp_attn_sparse", SPARSE, kw) == (xp.XP_ERR_SHAPE if bad else xp.XP_ERR_WORKSPACE), (where, os_)


# the bytes of each array that a call reads, from its sizes in test_step_host.py
READ = {"xp_kv_blocks": (BLOCKS, dict(cu=8, start=4, table=4)),
        "xp_attn_select": (SELECT, dict(cu=8, start=4, table=16, blocks=2 * 4 * 65)),
        "xp_attn_chunk": (CHUNK, dict(cu=8, start=4, table=16, cache=2 * 4 * 2 * 2176)),
        "xp_attn_sparse": (SPARSE, dict(cu=8, start=4, table=16, cache=2 * 4 * 2 * 2176))}
# and the array that it writes, with its bytes
WRITTEN = {"xp_kv_blocks": ("blocks", 2 * 4 * 65), "xp_attn_select": ("sel", 3 * 2 * 3 * 4), "xp_attn_chunk": ("out", 3 * 512),
           "xp_attn_sparse": ("out", 3 * 512)}


@pytest.mark.parametrize("name", list(READ))
def test_what_a_call_reads_is_not_written_over(name):
    base, read = READ[name]
    to, wide = WRITTEN[name]
    where = base[to].value
    for key, size in read.items():
        step = 16 if key in ("cache", "blocks") else 4
        first = size if size % step == 0 else size + step - size % step
        for off in (0, wide - wide % step - step, step - first):   # the last place that meets it, and the first
            assert call(name, base, {key: ctypes.c_void_p(where + off)}) == xp.XP_ERR_SHAPE, (key, off)
        if "ws" in base:                                       # just beside it: on to the workspace, which is too small
            for off in (wide + (-wide) % step, -first):
                assert call(name, base, {key: ctypes.c_void_p(where + off), "bytes": 0}) == xp.XP_ERR_WORKSPACE, (key, off)


@pytest.mark.parametrize("name,sizes", [("xp_attn_chunk", dict(rows=40, max_len=9000, cols=150)), ("xp_attn_sparse", dict(rows=1, keep=400, cols=150))])
def test_a_workspace_over_other_arrays_is_refused(name, sizes):
    base = READ[name][0]
    where = base["ws"].value
    d, rows = xp.kv_dims(2, 64, 64, 4), sizes["rows"]
    need = xp.xp_attn_chunk_workspace_bytes(d, 4, rows, 1, 9000) if "max_len" in sizes else xp.xp_attn_sparse_workspace_bytes(d, 4, rows, 400)
    assert need > 4096
    for key in ("q", "out", "cache", "table", "cu", "start") + (("sel",) if "keep" in sizes else ()):
        for off in (0, (need - 16) // 16 * 16):
            assert call(name, base, dict(sizes, bytes=need, **{key: ctypes.c_void_p(where + off)})) == xp.XP_ERR_SHAPE, (key, off)
        assert call(name, base, dict(sizes, bytes=need - 1, **{key: ctypes.c_void_p(where + (need + 15) // 16 * 16)})) == xp.XP_ERR_WORKSPACE, key
    assert call(name, base, dict(sizes, bytes=need, q=ctypes.c_void_p(where), out=ctypes.c_void_p(where))) == xp.XP_ERR_SHAPE


# ------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("kv,heads,dim", [(1, 1, 64), (2, 8, 128), (8, 32, 128), (8, 40, 128), (4, 80, 64), (16, 16, 256), (1024, 1024, 64)])
def test_one_workspace_for_every_step(kv, heads, dim):
    """The packed tokens' workspace never falls as a step grows; chosen blocks' stays below the size that xp.h names."""
    d = xp.kv_dims(kv, dim, 64, 4)
    rows, batches, lens = (1, 2, 3, 4, 5, 8, 9, 15, 33, 64, 65, 100, 300, 2000), (1, 2, 7, 30, 64, 65, 300), (0, 1, 64, 512, 513, 1024, 1025, 2048, 2049, 70000)
    size = {x: xp.xp_attn_chunk_workspace_bytes(d, heads, *x) for x in itertools.product(rows, batches, lens)}
    for i, axis in enumerate((rows, batches, lens)):
        for x in size:
            at = axis.index(x[i]) + 1
            if at < len(axis):
                assert 16 <= size[x] <= size[x[:i] + (axis[at],) + x[i + 1:]], x
    # 512 pieces of a block's rows (128 at 256 columns) and as many of sixteens: outputs, maxima, sums and factors
    # in fp32; the list of 256 cut units before them, 28 bytes each, to whole 256
    cut = 512 * ((128 if dim == 256 else 256) + 16) * (dim + 3) * 4 + 7424
    assert set(size.values()) == {16, cut} and round(cut / 1e6) == {64: 37, 128: 73, 256: 76}[dim]
    most = 1024 * (16 * dim + 48)
    for n in list(range(1, 40)) + [63, 64, 100, 127, 128, 129, 255, 256, 257, 2000]:
        for keep in list(range(1, 80)) + [100, 255, 256, 1000, 4097, 16384, 1 << 24]:
            assert 16 <= xp.xp_attn_sparse_workspace_bytes(d, heads, n, keep) <= most, (n, keep)
