"""Host side of a serving step's entry points at their edges (no GPU): an empty batch, outputs
over inputs, workspaces."""
import ctypes

import pytest

from fp4_routed_expert_xp_amd import xp

from test_step_host import PLAN, at, call


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
