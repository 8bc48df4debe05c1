"""GPU: a serving step over the 4-bit cache — pages and places from lengths, attention of
packed new tokens, block summaries, block selection, attention over chosen blocks — against
plain forms (step_ref.py, attn_ref.py). Whole numbers are compared exactly, attention within a
bound computed for each element from the definition (see attn_ref.attend)."""
import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref
import step_ref as step
from test_gpu_attn import DT, FLOOR, HALF, dev, dims_of, ends, filled, ints, on_device, tables

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------- pages and places
def run_plan(d, lens, want, table, free, count, rows):
    t = {"lens": ints(lens), "want": ints(want), "table": dev(table), "free": dev(free), "count": ints([count])}
    out = {n: torch.full((k,), 77, dtype=torch.int32, device="cuda")
           for n, k in (("cu", len(lens) + 1), ("start", len(lens)), ("lens_out", len(lens)), ("seq", rows), ("pos", rows))}
    out["slot"] = torch.full((rows,), 77, dtype=torch.int64, device="cuda")
    xp.xp_kv_plan(d, t["lens"], t["want"], t["table"], t["free"], t["count"], out["cu"], out["start"], out["lens_out"],
                  out["seq"], out["pos"], out["slot"])
    return t, out


def random_step(rng, batch, cols, page, longest, spare):
    lens = rng.integers(0, longest + 1, batch)
    want = np.where(rng.random(batch) < 0.4, rng.integers(0, 5, batch), rng.integers(0, longest, batch))
    held = -(-lens // page)
    need = int((-(-(lens + want) // page) - held).sum())
    pages = int(held.sum()) + max(need, 1) + 3
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((batch, cols), -1, dtype=np.int32)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(pages, -1, dtype=np.int32)
    n = min(pages - at, int(spare * need) + 1)
    free[:n] = order[at:at + n]
    return lens.tolist(), want.tolist(), table, free, n, pages


@pytest.mark.parametrize("batch,cols,page,longest,rows,spare", [
    (1, 3, 64, 60, 64, 1.0), (5, 9, 64, 250, 2000, 1.0), (64, 6, 192, 500, 20000, 1.0), (64, 6, 192, 500, 9000, 0.4),
    (1024, 4, 64, 100, 4096, 1.0), (1025, 4, 64, 100, 200000, 0.7), (2500, 3, 128, 150, 200000, 1.0), (70, 40, 64, 1200, 4096, 1.0),
    (70, 40, 64, 1200, 100000, 0.5), (3, 2, 64, 50, 0, 1.0)])
def test_plan_and_release(batch, cols, page, longest, rows, spare):
    rng = np.random.default_rng(batch + cols)
    lens, want, table, free, count, pages = random_step(rng, batch, cols, page, longest, spare)
    if batch > 4:
        want[1], want[2], lens[3] = -5, 2 ** 31 - 1, -2          # ask for nothing
    d = xp.kv_dims(1, 64, page, pages)
    t, out = run_plan(d, lens, want, table, free, count, rows)
    host = table.copy()
    cu, start, lens_out, seq, pos, slot, height = step.plan(lens, want, host, free, count, rows, page, pages)
    for name, x in (("cu", cu), ("start", start), ("lens_out", lens_out), ("seq", seq), ("pos", pos), ("slot", slot)):
        np.testing.assert_array_equal(out[name].cpu().numpy(), x, err_msg=name)
    np.testing.assert_array_equal(t["table"].cpu().numpy(), host)
    np.testing.assert_array_equal(t["free"].cpu().numpy(), free)
    assert t["count"].item() == height
    # all of it back: as it was
    xp.xp_kv_release(d, out["lens_out"], t["lens"], t["table"], t["free"], t["count"])
    np.testing.assert_array_equal(t["table"].cpu().numpy(), table)
    np.testing.assert_array_equal(t["free"].cpu().numpy(), free)
    assert t["count"].item() == count
    # some sequences end, some are cut, some keep what they have; entries that are no page are not put back
    keep = np.array(lens_out)
    keep[::3] = -1
    keep[1::3] = keep[1::3] // 2
    host = table.copy()
    host[0, 0] = pages
    t["table"].copy_(dev(host))
    stack = free.copy()
    height = step.release(lens_out, keep, host, stack, count, page, pages)
    xp.xp_kv_release(d, out["lens_out"], ints(keep.tolist()), t["table"], t["free"], t["count"])
    np.testing.assert_array_equal(t["table"].cpu().numpy(), host)
    np.testing.assert_array_equal(t["free"].cpu().numpy(), stack)
    assert t["count"].item() == height


def test_plan_in_place_lengths_and_a_stack_out_of_range():
    d = xp.kv_dims(2, 128, 64, 6)
    table, free = np.full((2, 4), -1, dtype=np.int32), np.arange(6, dtype=np.int32)
    for count, height in ((9, 6), (-3, 0), (2, 2)):
        lens, t = ints([0, 0]), dev(table)
        n, cu, start, seq, pos = ints([count]), ints([9] * 3), ints([9] * 2), ints([9] * 300), ints([9] * 300)
        slot = torch.full((300,), 9, dtype=torch.int64, device="cuda")
        xp.xp_kv_plan(d, lens, ints([70, 128]), t, dev(free), n, cu, start, lens, seq, pos, slot)
        host = table.copy()
        want = step.plan([0, 0], [70, 128], host, free, count, 300, 64, 6)
        assert cu.tolist() == want[0].tolist() and start.tolist() == [0, 0] and lens.tolist() == want[2].tolist()
        assert seq.tolist() == want[3].tolist() and pos.tolist() == want[4].tolist() and slot.tolist() == want[5].tolist()
        assert t.tolist() == host.tolist() and n.item() == want[6]
    # a stack that is full takes no more
    n, f, t = ints([6]), dev(free), dev(np.array([[5, 4, -1, 2]], dtype=np.int32))
    xp.xp_kv_release(d, ints([2 ** 31 - 1]), ints([64]), t, f, n)
    assert t.tolist() == [[5, -1, -1, -1]] and f.tolist() == free.tolist() and n.item() == 6


def test_plan_of_many_sequences():
    batch = 65535
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 129, batch)
    pages = 3 * batch
    order = rng.permutation(pages).astype(np.int32)
    table = np.where(np.arange(3) < -(-lens // 64)[:, None], order[:3 * batch].reshape(batch, 3), -1).astype(np.int32)
    free = rng.permutation(pages).astype(np.int32)
    d = xp.kv_dims(1, 64, 64, pages)
    want = rng.integers(0, 3, batch)
    t, out = run_plan(d, lens.tolist(), want.tolist(), table, free, pages, 60000)
    host = table.copy()
    got = step.plan(lens, want, host, free, pages, 60000, 64, pages)
    for name, x in zip(("cu", "start", "lens_out", "seq", "pos", "slot"), got):
        np.testing.assert_array_equal(out[name].cpu().numpy(), x, err_msg=name)
    np.testing.assert_array_equal(t["table"].cpu().numpy(), host)
    assert t["count"].item() == got[6]
    xp.xp_kv_release(d, out["lens_out"], t["lens"], t["table"], t["free"], t["count"])
    np.testing.assert_array_equal(t["table"].cpu().numpy(), table)
    np.testing.assert_array_equal(t["free"].cpu().numpy(), free)


# ---------------------------------------------------------------------- chunk
def run_chunk(c, buf, table, cu, start, q, scale, window=0, max_len=None, out=None):
    d = dims_of(c)
    if max_len is None:
        max_len = max(1, int(max(int(start[b]) + int(cu[b + 1] - cu[b]) for b in range(len(start)))))
    ws = torch.full((xp.xp_attn_chunk_workspace_bytes(d, q.shape[1], q.shape[0], len(start), max_len),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0) if out is None else out
    xp.xp_attn_chunk(d, q, buf, dev(table), dev(cu), ints([int(x) for x in start]), max_len, scale, out, ws, window=window)
    torch.cuda.synchronize()
    return out


def check_rows(want, got, v, p_step, tol, q_type):
    """Compare rows of float64 outputs within a bound; returns the largest share of it that was used."""
    assert np.array_equal(np.isnan(want), np.isnan(got))
    ok = ~np.isnan(want)
    # The weights are rounded by e (|e| <= p_step) in the products and in their sum: the output is off by
    # sum p e (v - out), at most p_step (sum p |v| + |out|); attend's bound holds the first part.
    tol = tol + p_step * np.abs(np.where(ok, want, 0.0)) + FLOOR[q_type]
    # fp16 holds at least 2^11 p (2^13 p, of a maximum that lags by up to 2^2, against a sum of at least 1): below its
    # normal range (steps of 2^-24) p rounds by up to 2^-25 / 2^11, in the products and in the sum
    tol = tol + 2.0 ** -35 * (np.nansum(np.abs(v), 0)[None, :] + len(v) * np.abs(np.where(ok, want, 0.0)))
    err = np.abs(got - want)
    assert (err[ok] <= tol[ok]).all(), float((err[ok] / tol[ok]).max())
    return float((err[ok] / tol[ok]).max()) if ok.any() else 0.0


def check_chunk(c, table, cu, start, q, out, scale, window=0, seqs=None):
    heads, group, cap = q.shape[1], q.shape[1] // c.kv, table.shape[1] * c.page
    qd, od = q.double().cpu().numpy(), out.double().cpu().numpy()
    worst = 0.0
    for b in range(len(start)) if seqs is None else seqs:
        n = int(cu[b + 1] - cu[b])
        if not n:
            continue
        at = np.arange(int(start[b]), int(start[b]) + n)
        m = int(min(max(at[-1] + 1, 0), cap))
        for h in range(c.kv):
            k, there = step.cached(c, table[b], h, m, "k")
            v, _ = step.cached(c, table[b], h, m, "v")
            rows = qd[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(n * group, c.dim)
            want, _, tol, _ = ref.attend(rows, k, v, np.repeat(at, group), scale, window, there, HALF[q.dtype], 2.0 ** -11)
            got = od[cu[b]:cu[b + 1], h * group:(h + 1) * group].reshape(n * group, c.dim)
            worst = max(worst, check_rows(want, got, v, 2.0 ** -11, tol, q.dtype))
    return worst


def some_q(rng, rows, heads, dim, ty, mag=2.0):
    return torch.from_numpy((mag * rng.normal(size=(rows, heads, dim))).astype(np.float32)).to(DT[ty]).cuda()


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("kv,group,dim,page,counts,start,window", [
    (1, 1, 64, 64, [1], [0], 0), (2, 4, 128, 192, [1, 0, 31, 33, 64, 130], [0, 5, 1, 64, 700, 63], 0),
    (2, 1, 64, 128, [257, 3], [0, 200], 0), (1, 5, 128, 64, [77, 20, 1], [10, 0, 300], 0),
    (1, 8, 256, 64, [40, 65], [0, 17], 0), (2, 2, 64, 64, [300, 70], [0, 100], 50), (1, 3, 128, 64, [190], [64], 1),
    (1, 2, 256, 128, [150], [90], 64), (1, 130, 64, 64, [3, 5], [0, 1], 0), (3, 2, 128, 64, [1, 1, 1], [0, 62, 500], 0)])
def test_chunk_lengths(kv, group, dim, page, counts, start, window, ty):
    rng = np.random.default_rng(sum(counts) + dim)
    cols = max(-(-(s + n) // page) for s, n in zip(start, counts)) + 1
    pages = len(counts) * cols + 2
    c = filled(rng, kv, dim, page, pages)
    table, cu = tables(rng, len(counts), cols, pages), ends(counts)
    q = some_q(rng, int(cu[-1]) + 3, kv * group, dim, ty)
    out = run_chunk(c, on_device(c), table, cu, start, q, dim ** -0.5, window)
    assert (out[int(cu[-1]):] == 3.0).all()                  # rows behind the last sequence stay
    check_chunk(c, table, cu, start, q, out, dim ** -0.5, window)


@pytest.mark.parametrize("kv,group,dim,page,counts,start,max_len", [
    (2, 8, 128, 256, [33], [9000], None), (1, 4, 64, 128, [5, 1], [12000, 40], None), (2, 4, 256, 64, [17], [5000], None),
    (1, 4, 128, 64, [300, 1, 1, 0, 2], [4000, 7000, 10, 9, 0], None), (1, 2, 128, 64, [3], [4000], 10),
    (4, 4, 128, 64, [520], [2900], None)])
def test_chunk_over_cut_sequences(kv, group, dim, page, counts, start, max_len):
    """Few rows behind many positions: sequences are cut and joined; a max_len that is too small leaves them whole."""
    rng = np.random.default_rng(len(counts) + dim)
    cols = max(-(-(s + n) // page) for s, n in zip(start, counts))
    pages = len(counts) * cols
    c = filled(rng, kv, dim, page, pages)
    table, cu = tables(rng, len(counts), cols, pages), ends(counts)
    q = some_q(rng, int(cu[-1]), kv * group, dim, "bf16")
    out = run_chunk(c, on_device(c), table, cu, start, q, dim ** -0.5, 0, max_len)
    check_chunk(c, table, cu, start, q, out, dim ** -0.5)


@pytest.mark.parametrize("batch", [64, 65, 200])
def test_chunk_many_sequences(batch):
    rng = np.random.default_rng(batch)
    kv, group, dim, page = 2, 2, 64, 64
    counts = rng.integers(0, 4, batch)
    counts[7], counts[batch - 1] = 150, 20
    start = rng.integers(0, 300, batch)
    start[3], start[batch - 1], counts[3] = 5000, 2500, 2
    cols = int(max(-(-(s + n) // page) for s, n in zip(start, counts)))
    c = filled(rng, kv, dim, page, 900)
    table = rng.integers(0, 900, (batch, cols)).astype(np.int32)     # pages shared: the call only reads them
    cu = ends(counts)
    q = some_q(rng, int(cu[-1]), kv * group, dim, "f16")
    out = run_chunk(c, on_device(c), table, cu, start, q, 0.125)
    check_chunk(c, table, cu, start, q, out, 0.125)


def test_chunk_places_that_are_not_there():
    """Missing pages are not seen, rows below position 0 see nothing, rows beyond the table what it has."""
    rng = np.random.default_rng(4)
    kv, dim, page, cols = 2, 128, 64, 4
    c = filled(rng, kv, dim, page, 12)
    table = np.array([[3, -1, 5, 12], [2 ** 31 - 1, 1, 0, 7], [4, 6, 8, 9], [-1, -1, -1, -1]], dtype=np.int32)
    counts, start = [40, 100, 90, 3], [180, -50, 200, 30]
    cu = ends(counts)
    q = some_q(rng, int(cu[-1]), kv * 2, dim, "bf16")
    for window in (0, 70):
        out = run_chunk(c, on_device(c), table, cu, start, q, 0.1, window)
        check_chunk(c, table, cu, start, q, out, 0.1, window)
        assert (out[cu[1]:cu[1] + 50] == 0).all() and (out[cu[3]:] == 0).all()
    # far beyond: a window there sees nothing, none sees all
    far = [2 ** 31 - 10, 2 ** 31 - 1, 256, -2 ** 31]
    for window in (0, 300):
        out = run_chunk(c, on_device(c), table, cu, far, q, 0.1, window, max_len=256)
        check_chunk(c, table, cu, far, q, out, 0.1, window)


@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_chunk_nan_only_where_seen(dim, group):
    rng = np.random.default_rng(dim)
    kv, page, cols = 1, 64, 5
    c = filled(rng, kv, dim, page, 5)
    table = np.arange(5, dtype=np.int32)[None]
    for p, g in ((70, 0), (200, dim // 32 - 1), (255, 0), (130, 1)):     # values of v that are not finite
        at = c.at(0, 0, p % 64, "v")[2][g]
        c.b[p // 64, 0, 0, at] = 127 if p != 130 else 255
    at = c.at(0, 0, 220 % 64, "k")[2][0]                                  # and a key
    c.b[3, 0, 0, at] = 127
    for p in range(256, 320):                                             # bytes behind the sequence are no values
        for which in "kv":
            c.b[4, 0, 0, c.at(0, 0, p % 64, which)[2]] = 127
    for window in (0, 33):
        q = some_q(rng, 256, group, dim, "f16")
        out = run_chunk(c, on_device(c), table, ends([256]), [0], q, dim ** -0.5, window)
        check_chunk(c, table, ends([256]), [0], q, out, dim ** -0.5, window)
        assert torch.isfinite(out[:70]).all()


@pytest.mark.parametrize("ty,mag", [("bf16", 1e30), ("bf16", 1e-30), ("f16", 1e-4), ("bf16", 3e38), ("f16", 6e4)])
def test_chunk_query_magnitudes(ty, mag):
    """Scores of any size: a row's weights are those of its largest scores alone, or all equal."""
    rng = np.random.default_rng(6)
    c = filled(rng, 1, 128, 64, 5)
    table = np.arange(5, dtype=np.int32)[None]
    q = torch.from_numpy(rng.uniform(-1, 1, size=(70, 4, 128))).mul(mag).to(DT[ty]).cuda()
    out = run_chunk(c, on_device(c), table, ends([70]), [230], q, 1.0 / mag if mag < 1 else 0.05)
    k, _ = step.cached(c, table[0], 0, 300, "k")
    v, _ = step.cached(c, table[0], 0, 300, "v")
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    qd = q.double().cpu().numpy()
    if mag < 1:
        check_chunk(c, table, ends([70]), [230], q, out, 1.0 / mag)
        return
    for i in range(70):
        s = qd[i] @ k[:231 + i].T * 0.05
        best = s.argmax(1)
        second = np.sort(s, 1)[:, -2]
        for h in range(4):
            # scores apart by more than any rounding of them (dim steps of 2^-24 of the sum of magnitudes) plus 60 weigh nothing
            slack = 0.05 * (np.abs(qd[i, h]) @ np.abs(k[:231 + i]).T).max() * 128 * 2.0 ** -24
            if s[h].max() - second[h] > 60 + 2 * slack:
                want = v[best[h]]
                assert (np.abs(got[i, h] - want) <= HALF[q.dtype] * np.abs(want) + 1e-12).all(), (i, h)


def test_chunk_infinite_query_stays_in_its_row():
    rng = np.random.default_rng(8)
    c = filled(rng, 1, 64, 64, 3)
    table = np.arange(3, dtype=np.int32)[None]
    q = some_q(rng, 40, 2, 64, "bf16")
    clean = run_chunk(c, on_device(c), table, ends([40]), [100], q, 0.125)
    q[5, 0, 3], q[9, 1, 0] = float("inf"), float("nan")
    out = run_chunk(c, on_device(c), table, ends([40]), [100], q, 0.125)
    other = torch.ones(40, 2, dtype=torch.bool, device="cuda")
    other[5, 0] = other[9, 1] = False
    assert torch.equal(out[other], clean[other]) and torch.isnan(out[9, 1]).all()


def test_chunk_rows_apart_on_q_another_stream_and_repeats():
    rng = np.random.default_rng(12)
    kv, group, dim, page = 2, 4, 128, 64
    counts, start = [200, 1, 40], [1000, 700, 0]
    c = filled(rng, kv, dim, page, 60)
    table, cu = tables(rng, 3, 20, 60), ends(counts)
    buf, heads = on_device(c), kv * group
    wide = some_q(rng, int(cu[-1]), 3 * heads, dim, "bf16")
    q = wide[:, heads:2 * heads]
    want = run_chunk(c, buf, table, cu, start, q.contiguous(), 0.09)
    side = torch.full((int(cu[-1]), 2 * heads, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    run_chunk(c, buf, table, cu, start, q, 0.09, out=side[:, heads:])
    assert torch.equal(side[:, heads:], want) and (side[:, :heads] == 5.0).all()
    inner = q.contiguous()
    run_chunk(c, buf, table, cu, start, inner, 0.09, out=inner)
    assert torch.equal(inner, want)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(5):
            assert torch.equal(run_chunk(c, buf, table, cu, start, q, 0.09), want)
    with pytest.raises(xp.XPError):
        run_chunk(c, buf, table, cu, start, q, 0.09, out=wide[:, heads + 1:2 * heads + 1])


# -------------------------------------------------------------- block summaries
@pytest.mark.parametrize("kv,dim,page,counts,start", [
    (1, 64, 64, [64], [0]), (3, 128, 192, [1, 0, 70, 300, 129, 1], [63, 5, 62, 1, 64, 126]), (2, 256, 128, [500, 63], [0, 0]),
    (8, 128, 64, [1] * 70, list(range(0, 140, 2))), (1, 64, 64, [130, 200], [-70, 100])])
def test_blocks(kv, dim, page, counts, start):
    rng = np.random.default_rng(kv + dim)
    batch, cols = len(counts), 9
    pages = batch * cols + 1
    c = filled(rng, kv, dim, page, pages)
    c.b[1] = rng.integers(0, 256, c.b[1].shape, dtype=np.uint8)            # any bytes: NaN and negative scales too
    for g in (0, dim // 32 - 1):                                           # the largest sums: all sixes times 448
        c.b[2, 0, 0, g * 1024:(g + 1) * 1024] = 0x77 if g else 0xff
        c.b[2, 0, 0, c.ng * 1024 + g * 64:c.ng * 1024 + (g + 1) * 64] = 126
    c.b[3, 0, 0] = 0
    table, cu = tables(rng, batch, cols, pages), ends(counts)
    table[0, :3] = [1, 2, 3][:len(table[0, :3])]
    table[-1, 0] = -1 if batch > 1 else table[-1, 0]
    d = dims_of(c)
    want = rng.integers(0, 256, xp.xp_kv_blocks_bytes(d), dtype=np.uint8)
    got = dev(want)
    xp.xp_kv_blocks(d, int(cu[-1]) + 5, dev(cu), ints(start), dev(table), on_device(c), got)
    step.summarise(c, want, cu, start, table)
    np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_blocks_of_chosen_sums():
    """Sums at the borders of k and ties of the rounding: one group's codes and scales by hand."""
    c = ref.Cache(1, 64, 64, 4)
    d = dims_of(c)
    for page, big in enumerate((127, 128, 254, 255)):
        for col in range(64):
            left = big if col == 0 else (col - 32) * 3
            for pos in range(64):
                codes, byte = c.get(page, 0, pos, "k")
                # scale byte 1 is 2^-9, so that codes are whole numbers of 2^-10: the most that is still wanted
                take = max(u for u in step.UNITS if 0 <= u <= left) if left >= 0 else min(u for u in step.UNITS if left <= u <= 0)
                codes[col] = step.UNITS.index(take)
                left -= take
                c.put(page, 0, pos, "k", codes, np.array([1, 1], dtype=np.uint8))
            assert left == 0
    want = np.zeros(xp.xp_kv_blocks_bytes(d), dtype=np.uint8)
    got = dev(want)
    table, cu, start = np.arange(4, dtype=np.int32)[None], ends([256]), [0]
    xp.xp_kv_blocks(d, 256, dev(cu), ints(start), dev(table), on_device(c), got)
    step.summarise(c, want, cu, start, table)
    assert [int(x) for x in want[4 * 64:]] == [0, 1, 1, 2]
    np.testing.assert_array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ selection
def check_select(c, table, cu, start, q, blocks, keep, sinks, recent):
    """Run it and compare every row's lists with the definition."""
    d, rows = dims_of(c), q.shape[0]
    sel = torch.full((rows, c.kv, keep), 99, dtype=torch.int32, device="cuda")
    xp.xp_attn_select(d, q, dev(cu), ints([int(x) for x in start]), dev(table), dev(blocks), sel, sinks=sinks, recent=recent)
    got = sel.cpu().numpy()
    assert (got[int(cu[-1]):] == 99).all()
    entries, tiles = c.pages * c.kv * (c.page // 64), c.page // 64
    codes, ks = blocks[:entries * c.dim].view(np.int8).reshape(entries, c.dim).astype(np.int64), blocks[entries * c.dim:]
    qd, group = q.double().cpu().numpy(), q.shape[1] // c.kv
    for b in range(len(start)):
        for r in range(cu[b], cu[b + 1]):
            p = min(int(start[b]) + int(r - cu[b]), table.shape[1] * c.page - 1)
            n = p // 64 + 1 if p >= 0 else 0
            page = table[b, np.arange(n) // tiles].astype(np.int64)
            there = (page >= 0) & (page < c.pages)
            for h in range(c.kv):
                e = np.where(there, (page * c.kv + h) * tiles + np.arange(n) % tiles, 0)
                s = step.scores(qd[r, h * group:(h + 1) * group], codes[e], ks[e])
                want = step.select(s, there, n, keep, sinks, recent)
                assert got[r, h].tolist() == want + [-1] * (keep - len(want)), (b, r, h)
    return sel


def random_blocks(rng, c, span=(5, 12)):
    entries = c.pages * c.kv * (c.page // 64)
    codes = np.clip(np.rint(30 * rng.normal(size=(entries, c.dim))), -127, 127).astype(np.int8)
    return np.concatenate([codes.view(np.uint8).reshape(-1), rng.integers(*span, entries).astype(np.uint8)])


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("kv,group,dim,page,counts,start,keep,sinks,recent", [
    (1, 1, 64, 64, [1], [0], 1, 0, 1), (2, 4, 128, 192, [1, 0, 5, 3, 1], [0, 5, 3000, 1021, 4000], 8, 1, 2),
    (1, 16, 64, 64, [4, 1], [2000, 64 * 9 - 1], 9, 0, 1), (3, 5, 256, 128, [2, 1], [5000, 700], 16, 2, 3),
    (1, 17, 128, 64, [3], [1500], 4, 1, 1), (1, 40, 64, 64, [2], [2500], 5, 0, 1), (2, 2, 128, 256, [2, 1], [-1, 9000], 3, 1, 2),
    (1, 8, 128, 64, [1, 1], [130000, 70000], 64, 1, 1), (8, 4, 128, 64, [1] * 66, list(range(0, 6600, 100)), 7, 0, 2)])
def test_select(kv, group, dim, page, counts, start, keep, sinks, recent, ty):
    rng = np.random.default_rng(sum(counts) + dim + keep)
    batch = len(counts)
    cols = max(-(-(s + n) // page) for s, n in zip(start, counts)) + 1
    c = ref.Cache(kv, dim, page, min(batch * cols, 400))
    table = rng.integers(0, c.pages, (batch, cols)).astype(np.int32)
    cu = ends(counts)
    q = some_q(rng, int(cu[-1]) + 2, kv * group, dim, ty)
    check_select(c, table, cu, start, q, random_blocks(rng, c), keep, sinks, recent)


def test_select_ties_missing_pages_and_odd_heads():
    rng = np.random.default_rng(2)
    c = ref.Cache(2, 64, 64, 50)
    table = rng.integers(0, 50, (2, 60)).astype(np.int32)
    table[0, 4:20], table[1, 50:] = -1, 50
    cu, start = ends([3, 4]), [3600, 60 * 64 - 2]             # the last rows lie beyond the table
    q = some_q(rng, 7, 4, 64, "f16")
    q[0, 0, 5], q[1, 1, 0], q[2], q[3, 0] = float("inf"), float("nan"), 0.0, 0.0
    q[4, 1] *= 2.0 ** -8                                       # a head of small steps beside a large one
    q[5, 0], q[5, 1] = 127.0 / 128, -127.0 / 128              # at the border of a step: 127 and just above it
    q[6, 0], q[6, 1] = 127.5 / 128, 1.0
    flat = random_blocks(rng, c)
    entries = c.pages * c.kv
    flat[:entries * 64] = np.tile(flat[:64], entries)         # every block the same: the lowest ones
    flat[entries * 64:] = 7
    for blocks in (flat, random_blocks(rng, c), random_blocks(rng, c, (0, 22)), np.zeros_like(flat)):
        check_select(c, table, cu, start, q, blocks, 12, 1, 2)
        check_select(c, table, cu, start, q, blocks, 3, 1, 2)  # nothing left to choose
        check_select(c, table, cu, start, q, blocks, 50, 0, 1) # more than have a page


def test_select_scales_far_apart():
    rng = np.random.default_rng(21)
    c = ref.Cache(1, 128, 64, 40)
    table = np.arange(40, dtype=np.int32)[None]
    q = some_q(rng, 6, 3, 128, "bf16")
    for i, e in enumerate((-120, -64, -20, 20, 60, 120)):
        q[i, 0] = (q[i, 0].double() * 2.0 ** e).to(torch.bfloat16)
    check_select(c, table, ends([6]), [2500], q, random_blocks(rng, c), 10, 1, 1)


# ------------------------------------------------------------- chosen blocks
def run_sparse(c, buf, table, cu, start, q, sel, scale, out=None):
    d = dims_of(c)
    ws = torch.full((xp.xp_attn_sparse_workspace_bytes(d, q.shape[1], q.shape[0], sel.shape[2]),), 255, dtype=torch.uint8,
                    device="cuda")
    out = torch.full_like(q, 3.0) if out is None else out
    xp.xp_attn_sparse(d, q, buf, dev(table), dev(cu), ints([int(x) for x in start]), sel, scale, out, ws)
    torch.cuda.synchronize()
    return out


def check_sparse(c, table, cu, start, q, sel, out, scale):
    heads, group, cap = q.shape[1], q.shape[1] // c.kv, table.shape[1] * c.page
    qd, od, lists = q.double().cpu().numpy(), out.double().cpu().numpy(), sel.cpu().numpy()
    worst = 0.0
    for b in range(len(start)):
        if cu[b + 1] == cu[b]:
            continue
        last = min(int(start[b]) + int(cu[b + 1] - cu[b]), cap)
        kv = [[step.cached(c, table[b], h, max(last, 0), w) for w in "kv"] for h in range(c.kv)]
        for r in range(cu[b], cu[b + 1]):
            at = min(int(start[b]) + int(r - cu[b]), cap - 1)
            for h in range(c.kv):
                (k, there), (v, _) = kv[h]
                p = [64 * int(j) + np.arange(64) for j in lists[r, h] if 0 <= j <= at // 64]
                p = np.concatenate(p) if p else np.zeros(0, dtype=np.int64)
                p = p[p <= at]
                p = p[there[p]]
                rows = qd[r, h * group:(h + 1) * group]
                want, _, tol, _ = ref.attend(rows, k[p], v[p], np.full(group, len(p)), scale, 0, None, HALF[q.dtype], 2.0 ** -11)
                worst = max(worst, check_rows(want, od[r, h * group:(h + 1) * group], v[p], 2.0 ** -11, tol, q.dtype))
    return worst


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("kv,group,dim,page,counts,start,keep", [
    (1, 1, 64, 64, [1], [0], 1), (2, 4, 128, 192, [1, 0, 5, 3, 1], [0, 5, 3000, 1021, 4000], 8),
    (1, 16, 64, 64, [4, 1], [2000, 575], 9), (3, 5, 256, 128, [2, 1], [5000, 700], 16), (1, 17, 128, 64, [3], [1500], 4),
    (1, 40, 64, 64, [2], [2500], 5), (1, 8, 128, 256, [1], [60000], 300), (4, 2, 256, 64, [2], [9000], 70),
    (2, 8, 64, 64, [1, 1], [20000, 100], 150), (8, 4, 128, 64, [1] * 70, list(range(0, 3500, 50)), 6)])
def test_sparse(kv, group, dim, page, counts, start, keep, ty):
    rng = np.random.default_rng(sum(counts) + dim + keep)
    batch = len(counts)
    cols = max(-(-(s + n) // page) for s, n in zip(start, counts)) + 1
    c = filled(rng, kv, dim, page, min(batch * cols, 300))
    table = rng.integers(0, c.pages, (batch, cols)).astype(np.int32)
    cu = ends(counts)
    q = some_q(rng, int(cu[-1]) + 2, kv * group, dim, ty)
    sel = np.full((q.shape[0], kv, keep), -1, dtype=np.int32)
    for b in range(batch):
        for r in range(cu[b], cu[b + 1]):
            n = (int(start[b]) + r - cu[b]) // 64 + 1
            for h in range(kv):
                some = np.sort(rng.permutation(n)[:keep])
                if h % 2 == 0 and n - 1 not in some:
                    some[-1] = n - 1
                sel[r, h, :len(some)] = some
    sel = dev(sel)
    out = run_sparse(c, on_device(c), table, cu, start, q, sel, dim ** -0.5)
    assert (out[int(cu[-1]):] == 3.0).all()
    check_sparse(c, table, cu, start, q, sel, out, dim ** -0.5)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sparse_odd_lists(dim):
    """Entries that name no block, blocks behind the row, twice the same, out of order, missing pages, none at all."""
    rng = np.random.default_rng(dim)
    c = filled(rng, 2, dim, 64, 20)
    table = rng.permutation(20)[:20].reshape(2, 10).astype(np.int32)
    table[0, 3], table[1, 2] = -1, 20
    counts, start = [4, 3], [500, 637]                        # rows beyond the table too
    cu = ends(counts)
    q = some_q(rng, 7, 6, dim, "bf16")
    sel = rng.integers(-3, 14, (7, 2, 11)).astype(np.int32)
    sel[0] = -1
    sel[1, 0] = 9                                             # behind its row
    sel[1, 1] = 3                                             # a page that is missing
    sel[2, 0] = 5                                             # eleven times the same
    sel[3, 0, 0], sel[3, 0, 1], sel[3, 0, 2] = 2 ** 31 - 1, -2 ** 31, 10
    # values that are not finite behind the row's position, and one that is seen
    c.b[int(table[0, 7]), :, 0, c.at(0, 0, 60, "v")[2]] = 127
    c.b[int(table[0, 7]), :, 0, c.at(0, 0, 60, "k")[2]] = 127
    c.b[int(table[1, 1]), 0, 0, c.at(0, 0, 5, "v")[2][0]] = 127
    sel[4, 0, :] = -1
    sel[4, 0, 4] = 1
    sel = dev(sel)
    out = run_sparse(c, on_device(c), table, cu, start, q, sel, 0.1)
    check_sparse(c, table, cu, start, q, sel, out, 0.1)
    assert (out[0] == 0).all() and torch.isnan(out[4, :3, :32]).all()
    # rows below position 0 see nothing
    out = run_sparse(c, on_device(c), table, cu, [-10, -2 ** 31], q, sel, 0.1)
    assert (out == 0).all()


@pytest.mark.parametrize("rows,keep", [(2, 400), (200, 5)])
def test_sparse_rows_apart_on_q_another_stream_and_repeats(rows, keep):
    rng = np.random.default_rng(rows)
    kv, group, dim, page = 2, 4, 128, 64
    c = filled(rng, kv, dim, page, 100)
    table, cu, start = rng.integers(0, 100, (1, 500)).astype(np.int32), ends([rows]), [26000]
    buf, heads = on_device(c), kv * group
    sel = dev(np.sort(rng.permutation(400)[:keep])[None, None].repeat(rows, 0).repeat(kv, 1).astype(np.int32))
    wide = some_q(rng, rows, 3 * heads, dim, "f16")
    q = wide[:, heads:2 * heads]
    want = run_sparse(c, buf, table, cu, start, q.contiguous(), sel, 0.09)
    side = torch.full((rows, 2 * heads, dim), 5.0, dtype=torch.float16, device="cuda")
    run_sparse(c, buf, table, cu, start, q, sel, 0.09, out=side[:, heads:])
    assert torch.equal(side[:, heads:], want) and (side[:, :heads] == 5.0).all()
    inner = q.contiguous()
    run_sparse(c, buf, table, cu, start, inner, sel, 0.09, out=inner)
    assert torch.equal(inner, want)
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(5):
            assert torch.equal(run_sparse(c, buf, table, cu, start, q, sel, 0.09), want)
    with pytest.raises(xp.XPError):
        run_sparse(c, buf, table, cu, start, q, sel, 0.09, out=wide[:, heads + 1:2 * heads + 1])


def test_sparse_over_all_blocks_is_the_whole_attention():
    rng = np.random.default_rng(30)
    kv, group, dim, page = 2, 4, 128, 128
    c = filled(rng, kv, dim, page, 30)
    table, cu, start = tables(rng, 2, 15, 30), ends([5, 3]), [1500, 200]
    q = some_q(rng, 8, kv * group, dim, "f16")
    sel = ints(list(range(30)))[None, None].expand(8, kv, 30).contiguous()
    out = run_sparse(c, on_device(c), table, cu, start, q, sel, 0.09)
    check_chunk(c, table, cu, start, q, out, 0.09)
