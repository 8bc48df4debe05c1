"""GPU: the calls of a serving step as they are used — together over several steps, captured and
replayed, on two streams, in a cache of more than 4 GiB — the row counts at which kernels change,
and refusals. Bounds are those of test_gpu_step.py; what two runs of the same numbers give is equal."""
import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref
import step_ref as step
from test_gpu_attn import dev, dims_of, ends, filled, ints, on_device, tables
from test_gpu_step import check_chunk, check_select, check_sparse, random_blocks, run_chunk, run_sparse, some_q

pytestmark = pytest.mark.gpu


# ------------------------------------------------ row counts where kernels change
@pytest.mark.parametrize("kv,group,dim,page,counts,start,keep,sinks,recent", [
    (8, 4, 128, 64, [70], [3000], 8, 1, 2), (4, 8, 64, 128, [129, 0, 3], [1000, 5, 200], 6, 0, 1),
    (16, 1, 256, 64, [33, 7], [500, 3], 4, 1, 1), (8, 2, 128, 192, [64], [5000], 9, 0, 2), (8, 4, 128, 64, [80], [900], 3, 1, 2),
    (8, 4, 64, 64, [64], [127000], 5, 1, 1), (8, 8, 256, 64, [65], [-10], 2, 0, 1), (16, 4, 64, 64, [13, 20, 1], [40000, 63, 20000], 7, 2, 2),
    (8, 3, 128, 64, [70], [3000], 8, 1, 2), (8, 4, 64, 64, [70], [140000], 6, 1, 1), (8, 4, 64, 64, [66], [9000], 70, 1, 1),
    (8, 4, 128, 64, [66], [5000], 64, 0, 1), (8, 1, 64, 64, [130], [4090], 63, 1, 3),
    (8, 4, 128, 64, [101], [3000], 8, 1, 2), (8, 8, 64, 128, [97, 0, 3], [1000, 5, 200], 6, 0, 1), (16, 1, 256, 64, [43, 7], [500, 3], 4, 1, 1),
    (8, 2, 128, 192, [100], [5000], 9, 0, 2), (8, 4, 64, 64, [99], [9000], 70, 1, 1), (8, 4, 128, 64, [100], [900], 3, 1, 2)])
def test_select_of_neighbouring_rows(kv, group, dim, page, counts, start, keep, sinks, recent):
    rng = np.random.default_rng(sum(counts) + dim + keep)
    batch = len(counts)
    cols = max(-(-(s + n) // page) for s, n in zip(start, counts)) + 1
    c = ref.Cache(kv, dim, page, min(batch * cols, 100))
    table = rng.integers(0, c.pages, (batch, cols)).astype(np.int32)
    table[rng.random((batch, cols)) < 0.1] = -1
    cu = ends(counts)
    q = some_q(rng, int(cu[-1]) + 3, kv * group, dim, "bf16")
    q[1] = 0.0                                                # all scores equal
    q[2, :, 5] = float("inf")
    check_select(c, table, cu, start, q, random_blocks(rng, c), keep, sinks, recent)


@pytest.mark.parametrize("kv,group,dim,rows,start,keep", [(8, 1, 128, 257, 100, 3), (4, 20, 64, 280, 50, 2), (2, 3, 256, 1030, 7, 2)])
def test_sparse_of_many_rows(kv, group, dim, rows, start, keep):
    rng = np.random.default_rng(rows)
    cols = -(-(start + rows) // 64)
    c = filled(rng, kv, dim, 64, cols)
    table, cu = tables(rng, 1, cols, cols), ends([rows])
    table[0, 1] = -1
    q = some_q(rng, rows + 2, kv * group, dim, "f16")
    sel = dev(rng.integers(-1, cols, (rows + 2, kv, keep)).astype(np.int32))
    out = run_sparse(c, on_device(c), table, cu, [start], q, sel, dim ** -0.5)
    assert (out[rows:] == 3.0).all()
    check_sparse(c, table, cu, [start], q, sel, out, dim ** -0.5)
    run_sparse(c, on_device(c), table, cu, [start], q, sel, dim ** -0.5, out=q)          # in place
    assert torch.equal(q[:rows], out[:rows])


@pytest.mark.parametrize("kv,group,dim,counts,start,window", [
    (2, 4, 128, [33, 1], [9000, 7000], 2500), (2, 4, 64, [520], [4000], 3001), (1, 2, 256, [130, 2], [5000, 64], 4500),
    (1, 8, 128, [5] * 70, [1200] * 70, 1100)])
def test_chunk_window_over_cut_sequences(kv, group, dim, counts, start, window):
    rng = np.random.default_rng(window)
    cols = max(-(-(s + n) // 64) for s, n in zip(start, counts))
    c = filled(rng, kv, dim, 64, 300)
    table = rng.integers(0, 300, (len(counts), cols)).astype(np.int32)
    table[0, cols // 2] = 300
    cu = ends(counts)
    q = some_q(rng, int(cu[-1]), kv * group, dim, "bf16")
    out = run_chunk(c, on_device(c), table, cu, start, q, dim ** -0.5, window)
    check_chunk(c, table, cu, start, q, out, dim ** -0.5, window, seqs=range(min(len(counts), 9)))


@pytest.mark.parametrize("left", [1, 16, 17, 31, 32, 33, 48])
@pytest.mark.parametrize("dim", [64, 256])
def test_chunk_rows_left_behind_whole_blocks(dim, left):
    rng = np.random.default_rng(left + dim)
    block = 128 if dim == 256 else 256
    counts, start = [block + left, left, 1], [1100, 500, 1500]
    c = filled(rng, 2, dim, 64, 100)
    table, cu = tables(rng, 3, 30, 100), ends(counts)
    q = some_q(rng, int(cu[-1]), 2, dim, "f16")
    check_chunk(c, table, cu, start, q, run_chunk(c, on_device(c), table, cu, start, q, 0.1), 0.1)


# ------------------------------------------------------------------- together
KV, GROUP, DIM, PAGE, BATCH, COLS, ROWS, KEEP = 2, 4, 128, 128, 4, 12, 160, 5


class Step:
    """The tensors of a server of BATCH sequences, and a step over them."""

    def __init__(self, pages, seed):
        rng = np.random.default_rng(seed)
        self.d = xp.kv_dims(KV, DIM, PAGE, pages)
        z = lambda *n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")
        self.lens, self.want, self.cap, self.keep = z(BATCH), z(BATCH), z(BATCH), z(BATCH)
        self.table, self.free, self.count = z(BATCH, COLS) - 1, dev(rng.permutation(pages).astype(np.int32)), ints([pages])
        self.cu, self.start, self.seq, self.pos, self.slot = z(BATCH + 1), z(BATCH), z(ROWS), z(ROWS), z(ROWS, t=torch.int64)
        self.cache = z(xp.xp_kv_bytes(self.d), t=torch.uint8)
        self.blocks = z(xp.xp_kv_blocks_bytes(self.d), t=torch.uint8)
        self.q, self.full, self.some = (z(ROWS, KV * GROUP, DIM, t=torch.bfloat16) for _ in range(3))
        self.k, self.v = (z(ROWS, KV, DIM, t=torch.bfloat16) for _ in "kv")
        self.sel = z(ROWS, KV, KEEP)
        most = COLS * PAGE
        self.ws = [z(n, t=torch.uint8) for n in (xp.xp_attn_chunk_workspace_bytes(self.d, KV * GROUP, ROWS, BATCH, most),
                                                 xp.xp_attn_sparse_workspace_bytes(self.d, KV * GROUP, ROWS, KEEP))]

    def fill(self, seed, want, cap):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.want.copy_(ints(want))
        self.cap.copy_(ints(cap))

    def run(self):
        xp.xp_kv_plan(self.d, self.lens, self.want, self.table, self.free, self.count, self.cu, self.start, self.lens, self.seq,
                      self.pos, self.slot)
        xp.xp_kv_append(self.d, self.k, self.v, self.cu, self.start, self.table, self.cache)
        xp.xp_kv_blocks(self.d, ROWS, self.cu, self.start, self.table, self.cache, self.blocks)
        xp.xp_attn_chunk(self.d, self.q, self.cache, self.table, self.cu, self.start, COLS * PAGE, 0.09, self.full, self.ws[0])
        xp.xp_attn_select(self.d, self.q, self.cu, self.start, self.table, self.blocks, self.sel, sinks=1, recent=2)
        xp.xp_attn_sparse(self.d, self.q, self.cache, self.table, self.cu, self.start, self.sel, 0.09, self.some, self.ws[1])

    def end(self):
        """Sequences are cut to cap positions."""
        torch.minimum(self.lens, self.cap, out=self.keep)
        xp.xp_kv_release(self.d, self.lens, self.keep, self.table, self.free, self.count)
        torch.minimum(self.lens, self.cap, out=self.lens)

    def all(self):
        return {n: t for n, t in vars(self).items() if isinstance(t, torch.Tensor)}


FAR = 10 ** 6
# what is asked for, and what sequences are cut to at the step's end
STEPS = [([150, 3, 0, 1], [FAR] * 4), ([1, 100, 50, 1], [FAR, FAR, 40, FAR]), ([129, 1, 1, 20], [FAR, 0, FAR, FAR]), ([140, 0, 9, 1], [FAR] * 4),
         ([1, 130, 1, 1], [FAR] * 4), ([150, 7, 1, 1], [FAR] * 4), ([160, 0, 0, 0], [FAR] * 4), ([1, 64, 70, 1], [5, FAR, FAR, 0]),
         ([1, 1, 1, 1], [FAR] * 4), ([500, 1, 1, 1], [FAR] * 4), ([1, 60, 1, 1], [0] * 4)]


def test_steps_together_against_the_definitions():
    s = Step(14, 3)
    c = ref.Cache(KV, DIM, PAGE, 14)
    c.b[...] = 0
    table, free, count, lens = s.table.cpu().numpy(), s.free.cpu().numpy(), 14, np.zeros(BATCH, dtype=np.int64)
    blocks = s.blocks.cpu().numpy()
    for i, (want, cap) in enumerate(STEPS):
        s.fill(i, want, cap)
        s.run()
        cu, start, lens_out, seq, pos, slot, count = step.plan(lens, want, table, free, count, ROWS, PAGE, 14)
        for got, x in ((s.cu, cu), (s.start, start), (s.lens, lens_out), (s.seq, seq), (s.pos, pos), (s.slot, slot), (s.table, table)):
            np.testing.assert_array_equal(got.cpu().numpy(), x)
        cu = cu.astype(np.int32)
        ref.append(c, s.k.double().cpu().numpy(), s.v.double().cpu().numpy(), cu, start, table)
        np.testing.assert_array_equal(s.cache.cpu().numpy(), c.b.reshape(-1))
        step.summarise(c, blocks, cu, start, table)
        np.testing.assert_array_equal(s.blocks.cpu().numpy(), blocks)
        n = int(cu[-1])
        check_chunk(c, table, cu, start, s.q, s.full, 0.09)
        sel = check_select(c, table, cu, start, s.q, blocks, KEEP, 1, 2)
        assert torch.equal(sel[:n], s.sel[:n])
        check_sparse(c, table, cu, start, s.q, s.sel, s.some, 0.09)
        # rows that see no more than KEEP blocks see the same either way
        few = (s.pos[:n] < 64 * KEEP) & (s.pos[:n] >= 0)
        # (half a step of bf16 each, 2^-8; weights rounded by 2^-11 in products and sums each, |v| < 6)
        torch.testing.assert_close(s.some[:n][few].float(), s.full[:n][few].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
        s.end()
        keep = np.minimum(lens_out, cap)
        count = step.release(lens_out, keep, table, free, count, PAGE, 14)
        lens = keep.astype(np.int64)
        np.testing.assert_array_equal(s.table.cpu().numpy(), table)
        np.testing.assert_array_equal(s.free.cpu().numpy()[:count], free[:count])
        assert s.count.item() == count
    assert count == 14


def test_steps_captured_and_replayed_beside_each_other():
    """Two graphs, each with its own tensors, replayed in turn with eager work between: every replay gives
    what the same calls give when they are not captured."""
    graphs = []
    for seed in (1, 2):
        s, twin = Step(20, seed), Step(20, seed)
        s.fill(0, [0] * 4, [FAR] * 4)
        s.run()                                               # nothing asked for; kernels are loaded
        s.end()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
            s.end()
        graphs.append((g, s, twin))
    for t in (graphs[0][2], graphs[1][2]):
        t.fill(0, [0] * 4, [FAR] * 4)
        t.run()
        t.end()
    for i, (want, cap) in enumerate(STEPS):
        for j, (g, s, twin) in enumerate(graphs):
            order = want if j == 0 else want[::-1]
            s.fill(2 * i + j, order, cap)
            twin.fill(2 * i + j, order, cap)
            g.replay()
            if i % 2:
                torch.cuda.synchronize()
            twin.run()
            twin.end()
        for g, s, twin in graphs:
            theirs = twin.all()
            for name, t in s.all().items():
                assert torch.equal(t, theirs[name]), (i, name)


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(9)
    c = filled(rng, 2, 128, 64, 200)
    buf = on_device(c)
    cases = []
    for counts, start in (([300, 1, 33], [3000, 5000, 10]), ([1, 1, 90], [9000, 100, 6000])):
        table = rng.integers(0, 200, (3, 160)).astype(np.int32)
        q = some_q(rng, sum(counts), 8, 128, "bf16")
        sel = dev(rng.integers(-1, 40, (sum(counts), 2, 20)).astype(np.int32))
        cases.append((table, ends(counts), start, q, sel))
    want = [(run_chunk(c, buf, *x[:4], 0.09), run_sparse(c, buf, *x, 0.09)) for x in cases]
    d, outs = dims_of(c), []
    streams = [torch.cuda.Stream() for _ in cases]
    held = [(dev(t), dev(cu), ints(st), q, sel, *(torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        xp.xp_attn_chunk_workspace_bytes(d, 8, len(q), 3, 9001), xp.xp_attn_sparse_workspace_bytes(d, 8, len(q), 20))))
        for t, cu, st, q, sel in cases]
    torch.cuda.synchronize()
    for _ in range(6):
        for h, s in zip(held, streams):
            with torch.cuda.stream(s):
                t, cu, st, q, sel, w0, w1 = h
                full, some = torch.empty_like(q), torch.empty_like(q)
                xp.xp_attn_chunk(d, q, buf, t, cu, st, 9001, 0.09, full, w0)
                xp.xp_attn_sparse(d, q, buf, t, cu, st, sel, 0.09, some, w1)
                outs.append((full, some))
    torch.cuda.synchronize()
    for i, (full, some) in enumerate(outs):
        assert torch.equal(full, want[i % 2][0]) and torch.equal(some, want[i % 2][1]), i


# ---------------------------------------------------------------- large caches
def test_pages_behind_4_gib():
    """The same pages at the end of a cache of 4.9 GB give what they give in a small one."""
    rng = np.random.default_rng(41)
    kv, dim, pages, n = 8, 128, 60, 70000
    c = filled(rng, kv, dim, 64, pages)
    small, d, big = on_device(c), dims_of(c), xp.kv_dims(kv, dim, 64, n)
    assert xp.xp_kv_bytes(big) > 2 ** 32 + small.numel()
    cache = torch.zeros(xp.xp_kv_bytes(big), dtype=torch.uint8, device="cuda")
    cache[-small.numel():] = small
    counts, start = [300, 1, 40], [900, 1200, 0]
    table, cu, st = tables(rng, 3, 20, 60), dev(ends(counts)), ints(start)
    rows = sum(counts)
    q = some_q(rng, rows, 2 * kv, dim, "bf16")
    got = []
    for dd, buf, t in ((d, small, dev(table)), (big, cache, dev(table + (n - pages)))):
        blocks = torch.zeros(xp.xp_kv_blocks_bytes(dd), dtype=torch.uint8, device="cuda")
        full, some, sel = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((rows, kv, 6), dtype=torch.int32, device="cuda")
        ws = [torch.zeros(k, dtype=torch.uint8, device="cuda") for k in (
            xp.xp_attn_chunk_workspace_bytes(dd, 2 * kv, rows, 3, 1300), xp.xp_attn_sparse_workspace_bytes(dd, 2 * kv, rows, 6))]
        xp.xp_kv_blocks(dd, 1300, dev(ends([1200, 0, 40])), ints([0, 0, 0]), t, buf, blocks)
        xp.xp_attn_chunk(dd, q, buf, t, cu, st, 1300, 0.09, full, ws[0])
        xp.xp_attn_select(dd, q, cu, st, t, blocks, sel)
        xp.xp_attn_sparse(dd, q, buf, t, cu, st, sel, 0.09, some, ws[1])
        held = pages * kv * dim
        got.append((full, some, sel, blocks[(dd.n_pages - pages) * kv * dim:][:held], blocks[-pages * kv:]))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    check_sparse(c, table, ends(counts)[:2], start[:1], q[:300], got[1][2][:300], got[1][1][:300], 0.09)


def test_places_behind_32_bits():
    page, n = 1 << 20, 5000
    d = xp.kv_dims(1, 64, page, n)
    free = np.arange(n, dtype=np.int32)
    table = np.array([[4998, -1, -1], [-1, -1, -1]], dtype=np.int32)
    lens, want = [page - 3, 0], [8, 2]
    t = dev(table)
    out = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (3, 2, 2, 12, 12)] + [torch.zeros(12, dtype=torch.int64, device="cuda")]
    xp.xp_kv_plan(d, ints(lens), ints(want), t, dev(free), ints([n]), *out)
    host = table.copy()
    got = step.plan(lens, want, host, free, n, 12, page, n)
    for x, y in zip(out, got):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
    assert max(got[5]) > 2 ** 32 and t.tolist() == host.tolist()


# -------------------------------------------------------------------- refusals
def test_tensors_that_do_not_fit_are_refused():
    s = Step(20, 5)
    s.fill(0, [100, 5, 1, 1], [FAR] * 4)
    s.run()
    s.end()
    torch.cuda.synchronize()
    before = {n: t.clone() for n, t in s.all().items()}
    h = dict(vars(s), ws0=s.ws[0], ws1=s.ws[1])
    calls = {
        "plan": lambda a: xp.xp_kv_plan(s.d, a["lens"], a["want"], a["table"], a["free"], a["count"], a["cu"], a["start"], a["keep"], a["seq"],
                                        a["pos"], a["slot"]),
        "release": lambda a: xp.xp_kv_release(s.d, a["lens"], a["keep"], a["table"], a["free"], a["count"]),
        "blocks": lambda a: xp.xp_kv_blocks(s.d, ROWS, a["cu"], a["start"], a["table"], a["cache"], a["blocks"]),
        "chunk": lambda a: xp.xp_attn_chunk(s.d, a["q"], a["cache"], a["table"], a["cu"], a["start"], 1000, 0.09, a["full"], a["ws0"]),
        "select": lambda a: xp.xp_attn_select(s.d, a["q"], a["cu"], a["start"], a["table"], a["blocks"], a["sel"]),
        "sparse": lambda a: xp.xp_attn_sparse(s.d, a["q"], a["cache"], a["table"], a["cu"], a["start"], a["sel"], 0.09, a["full"], a["ws1"])}
    used = {"plan": "lens want table free count cu start keep seq pos slot", "release": "lens keep table free count",
            "blocks": "cu start table cache blocks", "chunk": "q cache table cu start full ws0", "select": "q cu start table blocks sel",
            "sparse": "q cache table cu start sel full ws1"}
    for name, run in calls.items():
        for arg in used[name].split():
            t = h[arg]
            wrong = {"host": t.cpu(), "type": t.to(torch.float32 if t.dtype != torch.float32 else torch.int32)}
            if arg not in ("seq", "table"):                   # their lengths are the call's rows and sequences
                wrong["short"] = t[:0] if arg[:2] == "ws" else t[:-1] if t.dim() == 1 else t[:-1, :, :-1]
            if t.dim() == 1 and t.numel() > 1:
                wrong["apart"] = t.repeat(2)[::2]
            for kind, w in wrong.items():
                with pytest.raises((ValueError, TypeError, xp.XPError)):
                    run(dict(h, **{arg: w}))
                    pytest.fail("%s took %s (%s)" % (name, arg, kind))
        with pytest.raises((ValueError, TypeError, xp.XPError)):
            run(dict(h, table=s.table.t()))
    torch.cuda.synchronize()
    for n, t in s.all().items():
        assert torch.equal(t, before[n]), n


def test_select_over_the_longest_table():
    rng = np.random.default_rng(16)
    c = ref.Cache(2, 64, 1024, 90)
    table = rng.integers(0, 90, (2, 1024)).astype(np.int32)
    q = some_q(rng, 5, 6, 64, "bf16")
    check_select(c, table, ends([3, 2]), [2 ** 20 - 2, 1047000], q, random_blocks(rng, c), 500, 1, 2)
    d = dims_of(c)
    with pytest.raises(xp.XPError):
        xp.xp_attn_select(d, q, dev(ends([3, 2])), ints([0, 0]), dev(np.zeros((2, 1025), dtype=np.int32)),
                          dev(random_blocks(rng, c)), torch.zeros((5, 2, 5), dtype=torch.int32, device="cuda"))
