"""GPU: a serving step's calls at their edges — an empty batch, sequences of more than one round
of the plan with long runs of pages, a thousand sequences' attention, one workspace for steps of any size."""
import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import test_gpu_step as base
from test_gpu_attn import dev, dims_of, ends, filled, ints, on_device

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


# ---------------------------------------- more than a round of sequences, long runs of pages
@pytest.mark.parametrize("batch,cols,page,longest,rows,spare", [
    (1100, 24, 64, 700, 400000, 1.0),       # all are served
    (1100, 24, 64, 700, 400000, 0.97),      # the pool ends among those of the second round
    (1100, 24, 64, 700, 212000, 1.0),       # the rows end there
    (2100, 24, 64, 700, 10 ** 6, 1.0), (2100, 24, 64, 700, 10 ** 6, 0.7), (1025, 12, 128, 700, 400000, 1.0)])
def test_plan_and_release_of_many_sequences_with_long_runs(batch, cols, page, longest, rows, spare):
    base.test_plan_and_release(batch, cols, page, longest, rows, spare)


# ---------------------------------------------------------------------- attention
def test_chunk_of_a_thousand_sequences():
    """Single tokens beside a piece and a long context, which is cut."""
    rng = np.random.default_rng(1000)
    batch, kv, group, dim = 1000, 1, 4, 64
    counts, start = np.ones(batch, dtype=np.int64), rng.integers(0, 200, batch)
    counts[::50], counts[700], start[700], start[999] = 0, 300, 100, 9000
    c = filled(rng, kv, dim, 64, 300)
    table = rng.integers(0, 300, (batch, 142)).astype(np.int32)      # pages shared: the call only reads them
    cu = ends(counts)
    q = base.some_q(rng, int(cu[-1]) + 1, kv * group, dim, "bf16")
    out = base.run_chunk(c, on_device(c), table, cu, start, q, 0.125)
    assert (out[-1] == 3.0).all()
    base.check_chunk(c, table, cu, start, q, out, 0.125)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_workspace_for_steps_of_any_size(dim):
    """Chosen blocks over the size that suits every call, packed tokens over the largest step's: the bits of calls with their own."""
    rng = np.random.default_rng(dim + 1)
    kv, group = 2, 4
    c = filled(rng, kv, dim, 64, 80)
    d, buf, table = dims_of(c), on_device(c), rng.integers(0, 80, (1, 200)).astype(np.int32)
    sparse_ws = torch.full((1024 * (16 * dim + 48),), 255, dtype=torch.uint8, device="cuda")
    chunk_ws = torch.full((xp.xp_attn_chunk_workspace_bytes(d, kv * group, 300, 1, 12800),), 255, dtype=torch.uint8, device="cuda")
    for rows, keep in ((1, 190), (15, 40), (16, 64), (31, 64), (32, 64), (33, 7), (64, 64), (300, 3)):
        q, cu, start = base.some_q(rng, rows, kv * group, dim, "bf16"), ends([rows]), [12000]
        sel = dev(rng.integers(-1, 188, (rows, kv, keep)).astype(np.int32))
        out = torch.full_like(q, 3.0)
        xp.xp_attn_sparse(d, q, buf, dev(table), dev(cu), ints(start), sel, 0.09, out, sparse_ws)
        assert torch.equal(out, base.run_sparse(c, buf, table, cu, start, q, sel, 0.09)), rows
        out = torch.full_like(q, 3.0)
        xp.xp_attn_chunk(d, q, buf, dev(table), dev(cu), ints(start), 12000 + rows, 0.09, out, chunk_ws)
        assert torch.equal(out, base.run_chunk(c, buf, table, cu, start, q, 0.09)), rows
