"""Host side of a serving step's entry points at their edges (no GPU): an empty batch, outputs
over inputs, workspaces."""
import ctypes

import pytest

from fp4_routed_expert_xp_amd import xp

from test_step_host import PLAN, SPARSE, at, call


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
