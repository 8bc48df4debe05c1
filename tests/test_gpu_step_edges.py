"""GPU: a serving step's calls at their edges — an empty batch, sequences of more than one round
of the plan with long runs of pages."""
import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

from test_gpu_attn import dev, ints

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- empty batch
@pytest.mark.parametrize("rows", [0, 1, 256, 257, 5000])
def test_plan_without_sequences(rows):
    """No sequence, no row: cu is 0, every entry of the maps -1, the stack as it was; nothing behind the arrays."""
    d = xp.kv_dims(2, 128, 64, 6)
    full = lambda n, t=torch.int32: torch.full((n,), 77, dtype=t, device="cuda")
    free, count, cu, seq, pos, slot = dev(np.arange(6, dtype=np.int32)), ints([4]), full(3), full(rows + 2), full(rows + 2), full(
        rows + 2, torch.int64)
    empty, table = full(0), torch.zeros((0, 5), dtype=torch.int32, device="cuda")
    xp.xp_kv_plan(d, empty, empty, table, free, count, cu, empty, empty, seq[:rows], pos[:rows], slot[:rows])
    assert cu.tolist() == [0, 77, 77] and count.tolist() == [4] and free.tolist() == list(range(6))
    for t in (seq, pos, slot):
        assert t.tolist() == [-1] * rows + [77, 77]
    # the calls behind it see no row
    xp.xp_kv_release(d, empty, empty, table, free, count)
    assert count.tolist() == [4] and free.tolist() == list(range(6))


def test_plan_without_sequences_captured():
    d = xp.kv_dims(1, 64, 64, 3)
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")
    empty, table, free, count = z(0), torch.zeros((0, 2), dtype=torch.int32, device="cuda"), z(3), ints([3])
    cu, seq, pos, slot = z(1), z(9), z(9), z(9, torch.int64)
    run = lambda: xp.xp_kv_plan(d, empty, empty, table, free, count, cu, empty, empty, seq, pos, slot)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(3):
        for t in (cu, seq, pos, slot):
            t.fill_(50 + i)
        g.replay()
        torch.cuda.synchronize()
        assert cu.tolist() == [0] and seq.tolist() == [-1] * 9 and pos.tolist() == [-1] * 9 and slot.tolist() == [-1] * 9
