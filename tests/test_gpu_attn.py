"""GPU: the 4-bit cache (append, read, evict), attention over it and prompt attention,
against plain float64 forms (attn_ref.py). What the cache holds is compared byte for
byte; attention within a bound computed for each element from the definition (see
attn_ref.attend): half a step of the output type, one rounding of each probability
(fp16 in decode, the type of v in prompt), fp32 for everything else."""
import ctypes

import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# Below fp16's normal range its steps are 2^-24; bf16 has fp32's range
FLOOR = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ends(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def tables(rng, batch, cols, pages):
    assert pages >= batch * cols
    return rng.permutation(pages)[:batch * cols].reshape(batch, cols).astype(np.int32)


def dims_of(c):
    return xp.kv_dims(c.kv, c.dim, c.page, c.pages)


def on_device(c):
    t = torch.from_numpy(c.b.reshape(-1).copy()).cuda()
    assert t.numel() == xp.xp_kv_bytes(dims_of(c))
    return t


def filled(rng, kv, dim, page, pages):
    """A cache of quantised normal values everywhere (so stale bytes are there too)."""
    c = ref.Cache(kv, dim, page, pages, rng=rng)
    for at in (c.ng * 1024, c.ng * 2112):
        c.b[..., at:at + c.ng * 64] = rng.integers(0x26, 0x33, c.b.shape[:3] + (c.ng * 64,), dtype=np.uint8)
    return c


# ------------------------------------------------------------ append and read
@pytest.mark.parametrize("kv,dim,page", [(1, 64, 64), (3, 128, 192), (8, 128, 64), (2, 256, 128)])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_append_and_read(ty, kv, dim, page):
    rng = np.random.default_rng(11 + kv + dim)
    counts, start = [1, 0, 70, 3, 129], [0, 5, 62, page - 1, 1]
    cu = ends(counts)
    rows, cols = int(cu[-1]) + 4, 5               # four rows behind the last sequence
    pages = 5 * cols + 2
    table = tables(rng, 5, cols, pages)
    x = [torch.from_numpy(rng.normal(size=(rows, kv, dim)).astype(np.float32)) for _ in "kv"]
    x[0][:, :, 5] *= 20.0
    x[1][2] = torch.round(x[1][2] * 4) / 4        # quarters: with 6 in the group the midpoints themselves
    x[1][2, :, ::32] = 6.0
    x[0][3] *= 1e-4                               # the smallest scales
    x[0][4, :, 0:32] = 0.0
    x[1][5, 0, 7] = 30000.0                       # beyond the last scale
    x[0][6, 0, 33] = float("inf")
    x[1][7, 0, 1] = float("nan")
    x[1][8, 0, 40] = -float("inf")
    x = [t.to(DT[ty]) for t in x]
    host = [t.double().numpy() for t in x]
    c = ref.Cache(kv, dim, page, pages, rng=rng)
    buf = on_device(c)
    d = dims_of(c)
    xp.xp_kv_append(d, x[0].cuda(), x[1].cuda(), dev(cu), ints(start), dev(table), buf)
    torch.cuda.synchronize()
    ref.append(c, host[0], host[1], cu, start, table)
    np.testing.assert_array_equal(buf.cpu().numpy(), c.b.reshape(-1))

    k, v = (torch.full((rows, kv, dim), 7.0, dtype=DT[ty], device="cuda") for _ in "kv")
    xp.xp_kv_read(d, dev(cu), ints(start), dev(table), buf, k, v)
    for got, which in ((k, "k"), (v, "v")):
        got = got.double().cpu().numpy()
        assert (got[int(cu[-1]):] == 7.0).all()   # rows behind the last sequence stay
        for b in range(5):
            for r in range(cu[b], cu[b + 1]):
                p = start[b] + r - cu[b]
                for h in range(kv):
                    want = ref.values(*c.get(int(table[b, p // page]), h, p % page, which))
                    np.testing.assert_array_equal(got[r, h], want)


def test_append_places_it_cannot_reach_and_strided_rows():
    rng = np.random.default_rng(3)
    kv, dim, page, pages, cols = 2, 64, 64, 6, 2
    c = ref.Cache(kv, dim, page, pages, rng=rng)
    table = np.array([[0, -1], [pages, 3], [2147483647, 4]], dtype=np.int32)
    counts, start = [70, 70, 80], [0, 0, 60]
    cu = ends(counts)
    wide = torch.from_numpy(rng.normal(size=(int(cu[-1]), 3 * kv, dim)).astype(np.float32)).cuda()
    k, v = wide[:, kv:2 * kv], wide[:, 2 * kv:]            # views into rows of a fused projection
    assert k.stride(0) == 3 * kv * dim
    buf = on_device(c)
    xp.xp_kv_append(dims_of(c), k, v, dev(cu), ints(start), dev(table), buf)
    ref.append(c, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, start, table)
    np.testing.assert_array_equal(buf.cpu().numpy(), c.b.reshape(-1))
    # negative and far starts write nothing
    before = buf.clone()
    xp.xp_kv_append(dims_of(c), k[:5], v[:5], ints([0, 2, 4, 5]), ints([-3, 128, 2147483647]), dev(table), buf)
    assert torch.equal(before, buf)
    ko, vo = (torch.full((int(cu[-1]), 5, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    xp.xp_kv_read(dims_of(c), dev(cu), ints(start), dev(table), buf, ko[:, 1:3], vo[:, 2:4])
    ko, vo = ko.double().cpu().numpy(), vo.double().cpu().numpy()
    assert (ko[:, 0] == 9).all() and (ko[:, 3:] == 9).all() and (vo[:, :2] == 9).all() and (vo[:, 4:] == 9).all()
    for b in range(3):
        for r in range(cu[b], cu[b + 1]):
            p = start[b] + r - cu[b]
            page_id = table[b, p // page] if p < cols * page else -1
            for h in range(kv):
                want = np.zeros(dim) if not 0 <= page_id < pages else ref.values(*c.get(int(page_id), h, p % page, "k"))
                np.testing.assert_array_equal(ko[r, 1 + h], want)


# --------------------------------------------------------------------- decode
def run_decode(c, buf, table, lens, q, scale, window=0, q_rows=1, weights=None, max_len=None, out=None):
    d = dims_of(c)
    max_len = int(max(lens.max(), 1)) if max_len is None else max_len
    ws = torch.full((xp.xp_attn_decode_workspace_bytes(d, q.shape[1], q_rows, len(lens), max_len),), 255, dtype=torch.uint8,
                    device="cuda")
    out = torch.full_like(q, 3.0) if out is None else out
    xp.xp_attn_decode(d, q, buf, dev(table), ints(lens.tolist()), max_len, scale, out, ws, q_rows=q_rows, window=window,
                      weights=weights)
    torch.cuda.synchronize()
    return out


def check_decode(c, table, lens, q, out, scale, window=0, q_rows=1, base=None, weights=None):
    """Compare with the float64 form; returns the largest share of the bound that was used."""
    heads, group = q.shape[1], q.shape[1] // c.kv
    qd, od = q.double().cpu().numpy(), out.double().cpu().numpy()
    worst = 0.0
    for b, n in enumerate(lens):
        n = int(min(max(n, 0), table.shape[1] * c.page))
        for h in range(c.kv):
            k, there = c.rows(table[b], h, n, "k")
            v, _ = c.rows(table[b], h, n, "v")
            rows = qd[b * q_rows:(b + 1) * q_rows, h * group:(h + 1) * group].reshape(q_rows * group, c.dim)
            at = np.repeat(np.arange(n - q_rows, n), group)
            want, p, tol, rel = ref.attend(rows, k, v, at, scale, window, there, HALF[q.dtype], 2.0 ** -11)
            got = od[b * q_rows:(b + 1) * q_rows, h * group:(h + 1) * group].reshape(q_rows * group, c.dim)
            assert (np.isnan(want) == np.isnan(got)).all(), (b, h)
            # fp16 holds 2^15 p: below its normal range (steps of 2^-24) p rounds by up to 2^-25 / 2^15,
            # against a sum of at least 1 (the largest exponential)
            err = np.abs(got - want)
            tol = tol + FLOOR[q.dtype] + 2.0 ** -40 * np.nansum(np.abs(v), 0)[None, :]
            ok = ~np.isnan(want)
            assert (err[ok] <= tol[ok]).all(), (b, h, n, float((err[ok] / tol[ok]).max()))
            if ok.any():
                worst = max(worst, float((err[ok] / tol[ok]).max()))
            if weights is not None:
                # each probability: its score's and sum's error; then fp32 adds to the accumulator
                w, w0 = weights[b, h].double().cpu().numpy(), base[b, h].double().cpu().numpy()
                s = p.sum(0)
                t = (rel - 2.0 ** -11).max(initial=0.0) * s + (q_rows * group + 2) * 2.0 ** -24 * (s + np.abs(w0[:n])) + 1e-30
                assert (np.isnan(w[:n]) == np.isnan(s)).all()
                fine = ~np.isnan(s)
                assert (np.abs(w[:n] - w0[:n] - s)[fine] <= t[fine]).all(), (b, h, float((np.abs(w[:n] - w0[:n] - s)[fine] / t[fine]).max()))
                assert np.array_equal(w[n:], w0[n:])
    return worst


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("kv,group,dim,page,q_rows,window", [
    (2, 1, 64, 64, 1, 0), (2, 4, 128, 64, 1, 0), (1, 8, 256, 128, 1, 0), (3, 5, 64, 192, 1, 100), (2, 8, 128, 256, 4, 0),
    (1, 7, 128, 64, 3, 33), (1, 16, 64, 64, 4, 0), (1, 8, 256, 64, 5, 70), (2, 1, 128, 64, 17, 0), (1, 40, 64, 64, 2, 1),
    (1, 48, 128, 64, 2, 0)])
def test_decode_lengths(kv, group, dim, page, q_rows, window, ty):
    rng = np.random.default_rng(100 + kv + group + dim + q_rows)
    lens = np.array([0, 1, 2, 63, 64, 65, 127, 130, 200, 511, 512, 577], dtype=np.int32)
    cols = -(-577 // page)
    pages = len(lens) * cols + 1
    c = filled(rng, kv, dim, page, pages)
    table = tables(rng, len(lens), cols, pages)
    q = dev(rng.normal(size=(len(lens) * q_rows, kv * group, dim)) * 2.0, DT[ty])
    w = torch.rand(len(lens), kv, cols * page, device="cuda")
    w0 = w.clone()
    out = run_decode(c, on_device(c), table, lens, q, dim ** -0.5, window, q_rows, weights=w)
    worst = check_decode(c, table, lens, q, out, dim ** -0.5, window, q_rows, base=w0, weights=w)
    print("share of the bound: %.2f" % worst, flush=True)


@pytest.mark.parametrize("n,max_len,batch", [(4097, 4097, 1), (5000, 100000, 2), (3000, 10, 1), (1, 65536, 1),
                                             (0, 65536, 1)])
def test_decode_split_lengths(n, max_len, batch):
    """Contexts cut into many splits, and lengths beside the one the launch was sized for."""
    rng = np.random.default_rng(n)
    kv, dim, page = 2, 64, 64
    cols = max(1, -(-n // page))
    c = filled(rng, kv, dim, page, batch * cols)
    table = tables(rng, batch, cols, batch * cols)
    lens = np.array([n] + [max(n - 999, 0)] * (batch - 1), dtype=np.int32)
    q = dev(rng.normal(size=(batch, 8, dim)) * 3.0, torch.bfloat16)
    w = torch.zeros(batch, kv, cols * page, device="cuda")
    out = run_decode(c, on_device(c), table, lens, q, 0.125, max_len=max_len, weights=w)
    check_decode(c, table, lens, q, out, 0.125, base=torch.zeros_like(w), weights=w)


@pytest.mark.parametrize("batch,max_len", [(70, 12000), (64, 12000), (130, 100), (9, 12000)])
def test_decode_ragged_batches(batch, max_len):
    """One long sequence among many short and empty ones: cut and whole sequences in one launch,
    in batches of more and of fewer sequences than lanes of a wave."""
    rng = np.random.default_rng(batch)
    kv, dim, page = 1, 64, 64
    lens = rng.integers(0, 130, batch).astype(np.int32)
    lens[batch // 2], lens[batch - 1], lens[0] = 11000, 3300, 0
    cols = -(-11000 // page)
    c = filled(rng, kv, dim, page, 250)
    table = np.full((batch, cols), -1, dtype=np.int32)
    for b in range(batch):                                 # sequences may share pages that are only read
        n = -(-int(lens[b]) // page)
        table[b, :n] = rng.permutation(250)[:n]
    q = dev(rng.normal(size=(batch * 2, 3, dim)) * 2, torch.float16)
    out = run_decode(c, on_device(c), table, lens, q, 0.125, q_rows=2, max_len=max_len)
    check_decode(c, table, lens, q, out, 0.125, q_rows=2)


@pytest.mark.parametrize("dim,group,q_rows,n,window", [(128, 8, 5, 3000, 0), (64, 4, 9, 4100, 0), (256, 8, 3, 2500, 0),
                                                       (128, 8, 5, 5000, 2100)])
def test_decode_many_rows_over_cut_sequences(dim, group, q_rows, n, window):
    """More than sixteen rows a kv head over contexts cut into pieces, with weights."""
    rng = np.random.default_rng(n)
    kv, page = 2, 128
    cols = -(-n // page)
    c = filled(rng, kv, dim, page, 2 * cols)
    table = tables(rng, 2, cols, 2 * cols)
    lens = np.array([n, 777], dtype=np.int32)
    q = dev(rng.normal(size=(2 * q_rows, kv * group, dim)) * 2, torch.bfloat16)
    w = torch.rand(2, kv, cols * page, device="cuda")
    w0 = w.clone()
    out = run_decode(c, on_device(c), table, lens, q, dim ** -0.5, window, q_rows, weights=w)
    check_decode(c, table, lens, q, out, dim ** -0.5, window, q_rows, base=w0, weights=w)


@pytest.mark.parametrize("batch,longest", [(40, 300), (64, 17000), (64, 130)])
def test_decode_many_units(batch, longest):
    """More units than CUs: whole sequences in order of length, and one that is cut all the same."""
    rng = np.random.default_rng(batch + longest)
    kv, dim, page = 8, 64, 64
    lens = rng.integers(0, 130, batch).astype(np.int32)
    lens[17], lens[3] = longest, 0
    cols = -(-longest // page)
    c = filled(rng, kv, dim, page, 280)
    table = np.full((batch, cols), -1, dtype=np.int32)
    for b in range(batch):                                 # pages that are only read may be shared
        m = -(-int(lens[b]) // page)
        table[b, :m] = rng.permutation(280)[:m]
    q = dev(rng.normal(size=(batch, kv, dim)) * 2, torch.float16)
    out = run_decode(c, on_device(c), table, lens, q, 0.125)
    check_decode(c, table, lens, q, out, 0.125)


def test_windows_as_wide_as_an_int():
    """A window of 2^31 - 1 is none, also where queries lie before the first key."""
    rng = np.random.default_rng(77)
    c = filled(rng, 1, 64, 64, 8)
    table = tables(rng, 4, 2, 8)
    lens = np.array([1, 3, 7, 100], dtype=np.int32)
    q = dev(rng.normal(size=(4 * 6, 2, 64)), torch.bfloat16)
    buf = on_device(c)
    out = run_decode(c, buf, table, lens, q, 0.125, 2 ** 31 - 1, 6)
    check_decode(c, table, lens, q, out, 0.125, 0, 6)
    assert torch.equal(out, run_decode(c, buf, table, lens, q, 0.125, 0, 6))
    cu_q, cu_k = ends([9, 70]), ends([2, 70])
    q = dev(rng.normal(size=(79, 2, 64)), torch.float16)
    k, v = (dev(rng.normal(size=(72, 1, 64)), torch.float16) for _ in "kv")
    out, none = torch.empty_like(q), torch.empty_like(q)
    xp.xp_attn_prompt(q, k, v, dev(cu_q), dev(cu_k), 0.125, out, window=2 ** 31 - 1)
    xp.xp_attn_prompt(q, k, v, dev(cu_q), dev(cu_k), 0.125, none)
    check_prompt(q, k, v, cu_q, cu_k, out, 0.125)
    assert torch.equal(out, none)


def test_decode_lengths_out_of_range_are_clamped():
    rng = np.random.default_rng(8)
    c = filled(rng, 2, 64, 64, 6)
    table = tables(rng, 3, 2, 6)
    lens = np.array([-5, 128, 2000000000], dtype=np.int32)
    q = dev(rng.normal(size=(3, 4, 64)), torch.float16)
    out = run_decode(c, on_device(c), table, lens, q, 0.125, max_len=128)
    check_decode(c, table, lens, q, out, 0.125)
    assert (out[0] == 0).all() and (out[2] != 0).any()


def test_decode_missing_pages_are_not_seen():
    rng = np.random.default_rng(21)
    c = filled(rng, 2, 128, 64, 9)
    table = tables(rng, 3, 3, 9)
    table[0, 0], table[0, 2] = -1, 9
    table[1, :] = -1                                       # nothing is left of this one
    table[2, 1] = 1 << 30
    lens = np.array([190, 150, 192], dtype=np.int32)
    q = dev(rng.normal(size=(3, 8, 128)) * 2, torch.bfloat16)
    w = torch.zeros(3, 2, 192, device="cuda")
    out = run_decode(c, on_device(c), table, lens, q, 0.09, weights=w)
    check_decode(c, table, lens, q, out, 0.09, base=torch.zeros_like(w), weights=w)
    assert (out[1] == 0).all() and (w[1] == 0).all()


@pytest.mark.parametrize("q_rows,window", [(1, 0), (4, 0), (3, 20)])
def test_decode_nan_only_where_seen(q_rows, window):
    """NaN scales in stale bytes, outside the window, in later drafted tokens and in seen positions."""
    rng = np.random.default_rng(31)
    kv, dim, page = 2, 128, 64
    c = filled(rng, kv, dim, page, 8)
    table = tables(rng, 4, 2, 8)
    lens = np.array([70, 100, 40, 128], dtype=np.int32)
    nan_at = {0: [70, 75, 127], 1: [99, 98], 2: [39, 5], 3: [60]}  # behind the end; the last tokens; the last and an old one
    for b, places in nan_at.items():
        for p in places:
            for h in range(kv):
                tile = c.b[table[b, p // page], h, 0]
                for which in ("k", "v") if p >= lens[b] else ("v",):
                    tile[c.at(0, 0, p % 64, which)[2][1]] = 0x7f
    q = dev(rng.normal(size=(4 * q_rows, 8, dim)) * 2, torch.float16)
    out = run_decode(c, on_device(c), table, lens, q, 0.09, window, q_rows)
    check_decode(c, table, lens, q, out, 0.09, window, q_rows)
    assert not torch.isnan(out[:q_rows]).any()
    assert torch.isnan(out[2 * q_rows - 1]).any() and not torch.isnan(out[:, :, :32]).any()


def test_decode_nan_key_reaches_the_rows_that_see_it():
    rng = np.random.default_rng(32)
    c = filled(rng, 1, 64, 64, 2)
    table = tables(rng, 1, 2, 2)
    c.b[table[0, 0], 0, 0][c.at(0, 0, 10, "k")[2][0]] = 0x7f
    q = dev(rng.normal(size=(2, 4, 64)), torch.bfloat16)
    for window, nan in ((0, True), (20, False)):
        out = run_decode(c, on_device(c), table, np.array([100], dtype=np.int32), q, 0.1, window, 2)
        assert bool(torch.isnan(out).all()) == nan and bool(torch.isnan(out).any()) == nan


@pytest.mark.parametrize("ty,mag", [("bf16", 1e30), ("bf16", 1e-30), ("f16", 1e-4), ("bf16", 3e38), ("f16", 6e4)])
def test_decode_query_magnitudes(ty, mag):
    """bf16 reaches far beyond fp16; each row is scaled by its own power of two."""
    rng = np.random.default_rng(41)
    c = filled(rng, 1, 128, 64, 4)
    table = tables(rng, 1, 4, 4)
    q = rng.uniform(-1, 1, size=(3, 4, 128))
    q[1] *= mag
    q[2, 1] = 0.0
    q = dev(q, DT[ty])
    scale = 1.0 / mag if mag > 1 else 2.0
    out = run_decode(c, on_device(c), np.repeat(table, 3, 0), np.array([256, 250, 199], dtype=np.int32), q, scale)
    check_decode(c, np.repeat(table, 3, 0), np.array([256, 250, 199], dtype=np.int32), q, out, scale)


def test_decode_infinite_query_stays_in_its_row():
    rng = np.random.default_rng(42)
    c = filled(rng, 2, 64, 64, 3)
    table = tables(rng, 1, 3, 3)
    lens = np.array([150], dtype=np.int32)
    q = dev(rng.normal(size=(1, 8, 64)), torch.bfloat16)
    clean = run_decode(c, on_device(c), table, lens, q, 0.1)
    q[0, 2, 5] = float("inf")
    q[0, 5, 9] = float("nan")
    out = run_decode(c, on_device(c), table, lens, q, 0.1)
    rows = [0, 1, 3, 4, 6, 7]
    assert torch.equal(out[0, rows], clean[0, rows])
    assert torch.isnan(out[0, 5]).all()


def test_decode_strided_rows_another_stream_and_repeats():
    rng = np.random.default_rng(51)
    kv, dim, page = 2, 128, 64
    c = filled(rng, kv, dim, page, 60)
    table = tables(rng, 2, 30, 60)
    lens = np.array([1900, 1333], dtype=np.int32)
    wide = dev(rng.normal(size=(2, 12, dim)), torch.bfloat16)
    q = wide[:, 2:10]
    out = torch.full((2, 11, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    d, buf = dims_of(c), on_device(c)
    ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, 8, 1, 2, 1900), dtype=torch.uint8, device="cuda")
    t, n = dev(table), ints(lens.tolist())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xp.xp_attn_decode(d, q, buf, t, n, 1900, 0.09, out[:, 1:9], ws, stream=side)
    side.synchronize()
    check_decode(c, table, lens, q, out[:, 1:9], 0.09)
    assert (out[:, 0] == 5).all() and (out[:, 9:] == 5).all()
    first = out.clone()
    for _ in range(5):                                     # the same bits every time, whatever the workspace holds
        ws.random_(0, 256)
        xp.xp_attn_decode(d, q, buf, t, n, 1900, 0.09, out[:, 1:9], ws)
        assert torch.equal(out, first)


def test_captured_step_appends_attends_and_replays():
    """Two captured steps that share a workspace, replayed with eager work between, against eager calls."""
    rng = np.random.default_rng(61)
    kv, dim, page, batch, cols = 2, 64, 64, 3, 20
    c = filled(rng, kv, dim, page, batch * cols)
    d, buf, t = dims_of(c), on_device(c), dev(tables(rng, batch, cols, batch * cols))
    k, v = (dev(rng.normal(size=(batch, kv, dim)), torch.bfloat16) for _ in "kv")
    q = dev(rng.normal(size=(batch, 4, dim)), torch.bfloat16)
    start, cu = ints([1000, 3, 640]), ints([0, 1, 2, 3])
    n = start + 1
    w = torch.zeros(batch, kv, cols * page, device="cuda")
    ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, 4, 1, batch, 1280), dtype=torch.uint8, device="cuda")

    def step(out, wt):
        xp.xp_kv_append(d, k, v, cu, start, t, buf)
        xp.xp_attn_decode(d, q, buf, t, n, 1280, 0.125, out, ws, weights=wt)

    out_a, out_b = torch.empty_like(q), torch.empty_like(q)
    step(out_a, w.clone())
    torch.cuda.synchronize()
    graphs = []
    for out in (out_a, out_b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(out, w)
        graphs.append(g)
    for i in range(4):
        k.normal_()
        q.normal_()
        start += 1
        n += 1
        w.zero_()
        saved = buf.clone()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got, gw, after = [out_a.clone(), out_b.clone()], w.clone(), buf.clone()
        buf.copy_(saved)
        want, ww = torch.empty_like(q), torch.zeros_like(w)
        step(want, ww)
        step(want, ww)
        assert torch.equal(got[0], want) and torch.equal(got[1], want) and torch.equal(gw, ww) and torch.equal(after, buf)


# ---------------------------------------------------------------------- evict
def run_evict(c, buf, table, lens, w, keep, sinks, recent, dst, in_place=False):
    d = dims_of(c)
    kept = torch.full((len(lens), c.kv, keep), 77, dtype=torch.int32, device="cuda")
    n, wd, t = ints(lens.tolist()), dev(w), dev(table)
    n_out = n if in_place else torch.full_like(n, 55)
    w_out = wd if in_place else torch.full((len(lens), c.kv, dst.shape[1] * c.page), 3.0, device="cuda")
    xp.xp_kv_evict(d, buf, t, n, wd, keep, dev(dst), kept, n_out, w_out, sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), n_out.cpu().numpy(), w_out.cpu().numpy()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kv,dim,page,keep,sinks,recent", [
    (1, 64, 64, 1, 0, 0), (2, 128, 64, 70, 4, 16), (3, 64, 192, 200, 0, 64), (1, 256, 64, 64, 64, 0), (2, 64, 128, 50, 20, 30),
    (1, 64, 256, 2500, 4, 100)])
def test_evict(kv, dim, page, keep, sinks, recent, in_place):
    rng = np.random.default_rng(200 + keep)
    top = max(keep + 900, 300)
    lens = np.array([0, 1, keep - 1, keep, keep + 1, top // 2, top], dtype=np.int32)
    cols = -(-top // page)
    dcols = cols if in_place else -(-keep // page)
    pages = len(lens) * (cols + dcols) + 1
    c = filled(rng, kv, dim, page, pages)
    ids = rng.permutation(pages).astype(np.int32)
    table = ids[:len(lens) * cols].reshape(len(lens), cols)
    dst = table if in_place else ids[len(lens) * cols:len(lens) * (cols + dcols)].reshape(len(lens), dcols)
    w = (rng.random((len(lens), kv, cols * page)) ** 6).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = 0.0
    w[5, :, 10:40] = 0.125                                 # runs of equal weights at the border
    w[6, 0, ::7] = np.float32(-0.0)
    w[6, 0, 50:60] = np.nan
    w[5, 0, 100] = np.inf
    w[5, 0, 101:103] = -np.inf
    buf = on_device(c)
    kept, n_out, w_out = run_evict(c, buf, table, lens, w, keep, sinks, recent, dst, in_place)
    want = ref.Cache(kv, dim, page, pages)
    want.b[...] = c.b
    for b, n in enumerate(lens):
        m = min(int(n), keep)
        assert n_out[b] == m
        for h in range(kv):
            ids = ref.evict_list(w[b, h], int(n), keep, sinks, recent)
            np.testing.assert_array_equal(kept[b, h, :m], ids)
            assert (kept[b, h, m:] == -1).all()
            np.testing.assert_array_equal(w_out[b, h, :m].view(np.uint32), w[b, h, ids].view(np.uint32))
            end = min(int(n), w_out.shape[2])
            assert (w_out[b, h, m:end] == 0).all()
            np.testing.assert_array_equal(w_out[b, h, end:].view(np.uint32),
                                          (w[b, h, end:] if in_place else np.full(w_out.shape[2] - end, 3.0, np.float32)).view(np.uint32))
            for i, p in enumerate(ids):
                for which in ("k", "v"):
                    want.put(int(dst[b, i // page]), h, i % page, which, *c.get(int(table[b, p // page]), h, int(p) % page, which))
    np.testing.assert_array_equal(buf.cpu().numpy(), want.b.reshape(-1))


@pytest.mark.parametrize("n,keep", [(20000, 5000), (32768, 30000), (40001, 123)])
def test_evict_long(n, keep):
    """Positions chosen from long contexts, below and beyond what the kernel holds on chip."""
    rng = np.random.default_rng(n)
    page = 256
    cols = -(-n // page)
    c = filled(rng, 2, 64, page, 4)
    table = np.full((1, cols), -1, dtype=np.int32)         # the choice alone: nothing lies behind the table
    dst = np.full((1, -(-keep // page)), -1, dtype=np.int32)
    w = np.exp(rng.normal(size=(1, 2, cols * page)) * 8).astype(np.float32)
    w[rng.random(w.shape) < 0.2] = 1e-3
    w[0, 1] *= np.where(rng.random(cols * page) < 0.5, -1, 1).astype(np.float32)
    buf = on_device(c)
    kept, n_out, w_out = run_evict(c, buf, table, np.array([n], dtype=np.int32), w, keep, 4, 32, dst)
    for h in range(2):
        ids = ref.evict_list(w[0, h], n, keep, 4, 32)
        np.testing.assert_array_equal(kept[0, h], ids)
        np.testing.assert_array_equal(w_out[0, h, :keep], w[0, h, ids])
    np.testing.assert_array_equal(buf.cpu().numpy(), c.b.reshape(-1))


@pytest.mark.parametrize("kv,dim,ty", [(8, 64, "bf16"), (4, 128, "f32"), (2, 256, "f16")])
def test_append_and_read_many_rows(kv, dim, ty):
    """Enough rows for the form that takes 64 of them at a time, sequences beginning anywhere in a tile."""
    rng = np.random.default_rng(dim)
    counts = [9000, 0, 1, 70, 5000, 2300, 513]
    if kv == 2:
        counts[0] = 17000
    start = [3, 0, 63, 64, 100, 17, 0]
    cu, page = ends(counts), 192
    cols = -(-(max(a + b for a, b in zip(counts, start))) // page)
    used = [-(-(a + b) // page) for a, b in zip(counts, start)]
    pages = sum(used) + 1
    ids = rng.permutation(pages)
    table = np.full((len(counts), cols), -1, dtype=np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    table[0, 1] = -1                                       # a page that is missing
    rows = int(cu[-1]) + 30
    k, v = (torch.from_numpy(rng.normal(size=(rows, kv, dim)).astype(np.float32) * 3).to(DT[ty]) for _ in "kv")
    d = xp.kv_dims(kv, dim, page, pages)
    buf = torch.zeros(xp.xp_kv_bytes(d), dtype=torch.uint8, device="cuda")
    xp.xp_kv_append(d, k.cuda(), v.cuda(), dev(cu), ints(start), dev(table), buf)
    ko, vo = (torch.full((rows, kv, dim), 7.0, dtype=torch.float32, device="cuda") for _ in "kv")
    xp.xp_kv_read(d, dev(cu), ints(start), dev(table), buf, ko, vo)
    missing = np.zeros(rows, dtype=bool)
    missing[page - 3:2 * page - 3] = True
    missing = missing[:int(cu[-1])]
    for x, o in ((k, ko), (v, vo)):
        want = ref.values(*ref.quantise(x[:int(cu[-1])].double().numpy()))
        want[missing] = 0.0
        np.testing.assert_array_equal(o[:int(cu[-1])].double().cpu().numpy(), want)
        assert (o[int(cu[-1]):] == 7.0).all()
    # the bytes themselves: row by row through the small form, into a second cache
    buf2 = torch.zeros_like(buf)
    step = 400
    for b in range(len(counts)):
        for r in range(0, counts[b], step):
            n = min(step, counts[b] - r)
            s = slice(int(cu[b]) + r, int(cu[b]) + r + n)
            xp.xp_kv_append(d, k[s].cuda(), v[s].cuda(), ints([0, n]), ints([start[b] + r]), dev(table[b:b + 1]), buf2)
    assert torch.equal(buf, buf2)


def test_evict_missing_pages():
    """A kept position without a page moves as zeros; a destination without one takes nothing."""
    rng = np.random.default_rng(6)
    c = filled(rng, 1, 64, 64, 8)
    table = np.array([[0, -1, 2]], dtype=np.int32)
    dst = np.array([[5, 99]], dtype=np.int32)
    w = np.zeros((1, 1, 192), dtype=np.float32)
    w[0, 0, 60:130] = 1.0
    buf = on_device(c)
    kept, _, _ = run_evict(c, buf, table, np.array([192], dtype=np.int32), w, 70, 0, 0, dst)
    np.testing.assert_array_equal(kept[0, 0], np.arange(60, 130))
    want = ref.Cache(1, 64, 64, 8)
    want.b[...] = c.b
    zero = (np.zeros(64, dtype=np.uint8), np.zeros(2, dtype=np.uint8))
    for i in range(64):
        for which in ("k", "v"):
            want.put(5, 0, i, which, *(c.get(0, 0, 60 + i, which) if i < 4 else zero))
    np.testing.assert_array_equal(buf.cpu().numpy(), want.b.reshape(-1))


# --------------------------------------------------------------------- prompt
def check_prompt(q, k, v, cu_q, cu_k, out, scale, window=0):
    group = q.shape[1] // k.shape[1]
    qd, kd, vd, od = (t.double().cpu().numpy() for t in (q, k, v, out))
    worst = 0.0
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for h in range(q.shape[1]):
            kk, vv = (x[cu_k[b]:cu_k[b + 1], h // group] for x in (kd, vd))
            at = np.arange(nk - nq, nk)
            want, _, tol, _ = ref.attend(qd[cu_q[b]:cu_q[b + 1], h], kk, vv, at, scale, window, None, HALF[q.dtype],
                                         HALF[q.dtype])
            got = od[cu_q[b]:cu_q[b + 1], h]
            assert np.array_equal(np.isnan(want), np.isnan(got)), (b, h)
            inf = np.isinf(want)
            assert np.array_equal(want[inf], got[inf]), (b, h)
            ok = np.isfinite(want)
            # The weights are rounded by e (|e| <= p_step) in the products and in their sum: the output is off by
            # sum p e (v - out), at most p_step (sum p |v| + |out|); the bound so far holds the first part
            tol = tol + HALF[q.dtype] * np.abs(want)
            # fp16 probabilities below its normal range round by up to 2^-25
            tol = tol + FLOOR[q.dtype] * (1.0 + np.abs(np.where(np.isfinite(vv), vv, 0.0)).sum(0)[None, :])
            err = np.abs(got - want)
            assert (err[ok] <= tol[ok]).all(), (b, h, float((err[ok] / tol[ok]).max()))
            if ok.any():
                worst = max(worst, float((err[ok] / tol[ok]).max()))
    return worst


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("kv,group,dim,nq,prefix,window", [
    (1, 1, 64, [1], [0], 0), (2, 4, 128, [1, 0, 31, 33, 64, 130], [0, 0, 0, 0, 0, 0], 0), (2, 1, 64, [257, 3], [0, 200], 0),
    (1, 5, 128, [77, 20, 1], [10, 0, 300], 0), (1, 8, 256, [40, 65], [0, 17], 0), (2, 2, 64, [300, 70], [0, 100], 50),
    (1, 3, 128, [190], [64], 1), (1, 2, 256, [150], [0], 64), (1, 130, 64, [3, 5], [0, 1], 0),
    (1, 1, 128, [10, 12, 80], [-4, -12, -70], 0)])
def test_prompt_lengths(kv, group, dim, nq, prefix, window, ty):
    """Ragged prompts; prefixes of earlier keys; a negative prefix has fewer keys than queries, down to none."""
    rng = np.random.default_rng(300 + dim + group)
    nk = [a + p for a, p in zip(nq, prefix)]
    cu_q, cu_k = ends(nq), ends(nk)
    extra = 3
    q = dev(rng.normal(size=(cu_q[-1] + extra, kv * group, dim)) * 2, DT[ty])
    k, v = (dev(rng.normal(size=(max(int(cu_k[-1]), 1), kv, dim)), DT[ty]) for _ in "kv")
    out = torch.full_like(q, 4.0)
    xp.xp_attn_prompt(q, k, v, dev(cu_q), dev(cu_k), dim ** -0.5, out, window=window)
    torch.cuda.synchronize()
    worst = check_prompt(q, k, v, cu_q, cu_k, out, dim ** -0.5, window)
    assert (out[int(cu_q[-1]):] == 4.0).all()
    print("share of the bound: %.2f" % worst, flush=True)


def test_prompt_many_sequences():
    """More sequences than lanes of a wave, empty ones among them."""
    rng = np.random.default_rng(71)
    nq = rng.integers(0, 9, 150)
    nq[[0, 63, 64, 149]] = 0
    cu = ends(nq)
    q = dev(rng.normal(size=(cu[-1], 2, 64)), torch.bfloat16)
    k, v = (dev(rng.normal(size=(cu[-1], 1, 64)), torch.bfloat16) for _ in "kv")
    out = torch.empty_like(q)
    xp.xp_attn_prompt(q, k, v, dev(cu), dev(cu), 0.125, out)
    check_prompt(q, k, v, cu, cu, out, 0.125)


@pytest.mark.parametrize("dim,ty,window", [(64, "bf16", 0), (64, "f16", 90), (128, "bf16", 70), (128, "f16", 0)])
def test_prompt_many_workgroups(dim, ty, window):
    """More workgroups than take the form for few of them: ragged prompts with prefixes, values that are
    not finite behind and before what rows see."""
    rng = np.random.default_rng(400 + dim)
    nq, prefix, kv, group = [150, 129, 0, 64, 1], [0, 70, 5, 0, 100], 64, 2
    nk = [a + b for a, b in zip(nq, prefix)]
    cu_q, cu_k = ends(nq), ends(nk)
    assert ((cu_q[-1] * group + 127) // 128 + len(nq)) * kv > 512
    q = dev(rng.normal(size=(cu_q[-1] + 2, kv * group, dim)) * 2, DT[ty])
    k, v = (rng.normal(size=(cu_k[-1], kv, dim)) for _ in "kv")
    v[100, :, 3], v[130, 5, 7], v[20, 6, 1] = np.nan, np.inf, -np.inf     # first sequence
    v[cu_k[1] + 190, 9, :], k[cu_k[1] + 180, 10, 2] = np.nan, np.nan      # near the second's end
    k, v = dev(k, DT[ty]), dev(v, DT[ty])
    out = torch.full_like(q, 4.0)
    xp.xp_attn_prompt(q, k, v, dev(cu_q), dev(cu_k), dim ** -0.5, out, window=window)
    worst = check_prompt(q, k, v, cu_q, cu_k, out, dim ** -0.5, window)
    assert (out[int(cu_q[-1]):] == 4.0).all()
    assert torch.isfinite(out[:20].float()).all()
    print("share of the bound: %.2f" % worst, flush=True)


@pytest.mark.parametrize("ty", ["bf16", "f16"])
def test_prompt_what_a_row_does_not_see(ty):
    """NaN and infinities in later positions, outside the window and in the next sequence stay away."""
    rng = np.random.default_rng(81)
    nq = [90, 40]
    cu = ends(nq)
    k, v = (rng.normal(size=(130, 1, 64)) for _ in "kv")
    q = rng.normal(size=(130, 2, 64))
    v[70, 0, 3], v[71, 0, 3], v[60, 0, 10], v[75, 0, 40] = np.inf, -np.inf, -np.inf, np.nan
    v[90, 0, 7] = np.nan
    v[129, 0, 8] = np.inf
    k[80, 0, 1] = np.nan
    k[128, 0, 2] = np.nan
    for window in (0, 12):
        t = [dev(x, DT[ty]) for x in (q, k, v)]
        out = torch.empty_like(t[0])
        xp.xp_attn_prompt(*t, dev(cu), dev(cu), 0.125, out, window=window)
        check_prompt(*t, cu, cu, out, 0.125, window)
        o = out.float()
        assert torch.isfinite(o[:60]).all() and not torch.isnan(o[:71]).any() and torch.isnan(o[80:90 if not window else 90]).any()


def test_prompt_infinite_scores():
    """Keys with infinities: rows that meet them hold what the formula gives (NaN), the others do not change."""
    rng = np.random.default_rng(82)
    q, k, v = (rng.normal(size=(100, 1, 64)) for _ in "qkv")
    t = [dev(x, torch.bfloat16) for x in (q, k, v)]
    cu = ends([100])
    clean = torch.empty_like(t[0])
    xp.xp_attn_prompt(*t, dev(cu), dev(cu), 0.125, clean)
    t[1][50, 0, 3] = float("nan")
    out = torch.empty_like(clean)
    xp.xp_attn_prompt(*t, dev(cu), dev(cu), 0.125, out)
    assert torch.equal(out[:50], clean[:50]) and torch.isnan(out[50:]).all()


def test_prompt_strided_captured_and_pieces():
    """A fused projection's views, a captured graph, and a prompt in two pieces through the cache's reader."""
    rng = np.random.default_rng(91)
    kv, group, dim, n = 2, 3, 128, 200
    fused = dev(rng.normal(size=(n, kv * (group + 2), dim)), torch.bfloat16)
    q, k, v = fused[:, :kv * group], fused[:, kv * group:kv * (group + 1)], fused[:, kv * (group + 1):]
    out = torch.zeros(n, kv * group + 1, dim, dtype=torch.bfloat16, device="cuda")[:, 1:]
    cu = dev(ends([n]))
    xp.xp_attn_prompt(q, k, v, cu, cu, 0.1, out)
    check_prompt(q, k, v, ends([n]), ends([n]), out, 0.1)
    piece = torch.empty(60, kv * group, dim, dtype=torch.bfloat16, device="cuda")
    xp.xp_attn_prompt(q[140:], k, v, dev(ends([60])), cu, 0.1, piece)
    check_prompt(q[140:], k, v, ends([60]), ends([n]), piece, 0.1)
    g = torch.cuda.CUDAGraph()
    replayed = torch.empty_like(q.contiguous())
    with torch.cuda.graph(g):
        xp.xp_attn_prompt(q, k, v, cu, cu, 0.1, replayed)
    for _ in range(3):
        fused.normal_()
        g.replay()
        torch.cuda.synchronize()
        xp.xp_attn_prompt(q, k, v, cu, cu, 0.1, out)
        assert torch.equal(replayed, out)


# ------------------------------------------------------------ the set together
def test_projections_prompt_cache_eviction_and_steps():
    """A layer's attention as it is served: FP8 projections, the prompt, its rows into the cache,
    a look back with weights, an eviction in place, and steps whose o projection reads bf16 rows."""
    rng = np.random.default_rng(1)
    hidden, heads, kv, dim, page = 256, 4, 2, 64, 64
    nq = [150, 90]
    cu = ends(nq)
    n_out = (heads + 2 * kv) * dim

    def fp8(n, k):
        w = torch.from_numpy(rng.normal(size=(n, k)).astype(np.float32) * 8).to(torch.float8_e4m3fn).cuda()
        packed = torch.empty(xp.xp_fp8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
        xp.xp_fp8_pack(w.view(torch.uint8), packed)
        s = torch.full(((n + 127) // 128, k // 128), 2.0 ** -7, device="cuda")
        return packed, s

    qkv_w, o_w = fp8(n_out, hidden), fp8(hidden, heads * dim)

    def project(x):
        y = torch.empty(x.shape[0], n_out, device="cuda")
        xp.xp_fp8_rows(x.shape[0], n_out, hidden, x, *qkv_w, y)
        y = y.view(x.shape[0], heads + 2 * kv, dim)
        return y[:, :heads].to(torch.bfloat16), y[:, heads:heads + kv], y[:, heads + kv:]

    x = dev(rng.normal(size=(int(cu[-1]), hidden)), torch.bfloat16)
    q, k, v = project(x)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    xp.xp_attn_prompt(q, k.to(torch.bfloat16), v.to(torch.bfloat16), dev(cu), dev(cu), 0.125, out)
    check_prompt(q, k.to(torch.bfloat16), v.to(torch.bfloat16), cu, cu, out, 0.125)

    cols = 4
    c = ref.Cache(kv, dim, page, 2 * cols, rng=rng)
    table = tables(rng, 2, cols, 2 * cols)
    d, buf, t = dims_of(c), on_device(c), dev(table)
    xp.xp_kv_append(d, k, v, dev(cu), ints([0, 0]), t, buf)    # fp32 rows, straight from the projection
    ref.append(c, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, [0, 0], table)
    np.testing.assert_array_equal(buf.cpu().numpy(), c.b.reshape(-1))

    lens = ints(nq)
    w = torch.zeros(2, kv, cols * page, device="cuda")
    back = torch.cat([q[cu[b + 1] - 8:cu[b + 1]] for b in range(2)])
    ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, heads, 8, 2, 256), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(back)
    xp.xp_attn_decode(d, back, buf, t, lens, 256, 0.125, o, ws, q_rows=8, weights=w)
    check_decode(c, table, np.array(nq), back, o, 0.125, 0, 8, base=torch.zeros_like(w), weights=w)

    keep = 100
    kept = torch.empty(2, kv, keep, dtype=torch.int32, device="cuda")
    wh = w.cpu().numpy()
    xp.xp_kv_evict(d, buf, t, lens, w, keep, t, kept, lens, w, sinks=2, recent=16)
    assert lens.tolist() == [100, 90]
    old = ref.Cache(kv, dim, page, 2 * cols)
    old.b[...] = c.b
    for b in range(2):
        for h in range(kv):
            ids = ref.evict_list(wh[b, h], nq[b], keep, 2, 16)
            np.testing.assert_array_equal(kept[b, h, :len(ids)].cpu().numpy(), ids)
            for i, p in enumerate(ids):
                for which in ("k", "v"):
                    c.put(int(table[b, i // page]), h, i % page, which, *old.get(int(table[b, p // page]), h, int(p) % page, which))
    np.testing.assert_array_equal(buf.cpu().numpy(), c.b.reshape(-1))

    for step in range(3):
        x = dev(rng.normal(size=(2, hidden)), torch.bfloat16)
        q, k, v = project(x)
        xp.xp_kv_append(d, k, v, ints([0, 1, 2]), lens, t, buf)
        ref.append(c, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 1, 2], lens.tolist(), table)
        lens += 1
        o, w0 = torch.empty(2, heads, dim, dtype=torch.bfloat16, device="cuda"), w.clone()
        xp.xp_attn_decode(d, q, buf, t, lens, 256, 0.125, o, ws, weights=w)
        check_decode(c, table, lens.cpu().numpy(), q, o, 0.125, base=w0, weights=w)
        y = torch.empty(2, hidden, device="cuda")
        xp.xp_fp8_rows(2, hidden, heads * dim, o, *o_w, y)
        assert torch.isfinite(y).all() and (y != 0).any()


def test_refusals_on_device_tensors():
    d = xp.kv_dims(2, 64, 64, 4)
    buf = torch.zeros(xp.xp_kv_bytes(d), dtype=torch.uint8, device="cuda")
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    t, cu, st = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), ints([0, 3]), ints([0])
    for bad in (x.double(), x[:, :1], x.transpose(1, 2), x[..., ::2], x[:2]):
        with pytest.raises(ValueError):
            xp.xp_kv_append(d, x, bad, cu, st, t, buf)
    with pytest.raises(ValueError):
        xp.xp_kv_append(d, x, x, cu.long(), st, t, buf)
    with pytest.raises(ValueError):
        xp.xp_kv_append(d, x, x, cu, st, t, buf[:-1])
    with pytest.raises(ValueError):
        xp.xp_kv_append(d, x, x, cu[:1], st, t, buf)
    with pytest.raises(ValueError):
        xp.xp_kv_append(d, x, x, cu, st, t.view(-1), buf)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(xp.xp_attn_decode_workspace_bytes(d, 4, 1, 1, 128), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        xp.xp_attn_decode(d, q.float(), buf, t, st, 128, 1.0, q.float(), ws)
    with pytest.raises(ValueError):
        xp.xp_attn_decode(d, q, buf, t, st, 128, 1.0, q.half(), ws)
    with pytest.raises(ValueError):
        xp.xp_attn_decode(d, q, buf, t, st, 128, 1.0, q.clone(), ws, weights=torch.zeros(1, 2, 127, device="cuda"))
    with pytest.raises(xp.XPError) as e:
        xp.xp_attn_decode(d, q, buf, t, st, 128, 1.0, q.clone(), ws[:0])
    assert e.value.status in (xp.XP_ERR_WORKSPACE, xp.XP_ERR_NULL)
    with pytest.raises(xp.XPError):
        xp.xp_attn_decode(d, q, buf, t, st, 128, -1.0, q.clone(), ws)
    with pytest.raises(ValueError):
        xp.xp_attn_prompt(q, x, x.half(), cu, cu, 1.0, q.clone())


def test_out_on_q_and_beside_it():
    """out may be q itself (without weights), and rows of one wider buffer may hold both beside each other."""
    rng = np.random.default_rng(17)
    kv, dim, page, n = 2, 64, 64, 3000
    c = filled(rng, kv, dim, page, 120)
    table = tables(rng, 2, 47, 94)
    d, buf, t = dims_of(c), on_device(c), dev(table)
    for lens in ([n, 2900], [100, 40]):                    # cut and whole
        size, ln = max(lens), ints(lens)
        ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, 8, 3, 2, size), dtype=torch.uint8, device="cuda")
        wide = dev(rng.normal(size=(6, 16, dim)), torch.bfloat16)
        q, o = wide[:, 3:11].clone(), torch.empty(6, 8, dim, dtype=torch.bfloat16, device="cuda")
        xp.xp_attn_decode(d, q, buf, t, ln, size, 0.125, o, ws, q_rows=3)
        xp.xp_attn_decode(d, q, buf, t, ln, size, 0.125, q, ws, q_rows=3)
        assert torch.equal(q, o)
        xp.xp_attn_decode(d, wide[:, :8], buf, t, ln, size, 0.125, wide[:, 8:], ws, q_rows=3,
                          weights=torch.zeros(2, kv, 47 * page, device="cuda"))
        xp.xp_attn_decode(d, wide[:, :8], buf, t, ln, size, 0.125, o, ws, q_rows=3)
        assert torch.equal(wide[:, 8:], o)
        for w in (None, torch.zeros(2, kv, 47 * page, device="cuda")):
            with pytest.raises(xp.XPError):
                xp.xp_attn_decode(d, wide[:, :8], buf, t, ln, size, 0.125, wide[:, 7:15], ws, q_rows=3, weights=w)
        with pytest.raises(xp.XPError):
            xp.xp_attn_decode(d, q, buf, t, ln, size, 0.125, q, ws, q_rows=3, weights=torch.zeros(2, kv, 47 * page, device="cuda"))
    cu = dev(ends([150, 61]))
    for group, heads_kv in ((2, 2), (2, 100)):             # both forms
        wide = dev(rng.normal(size=(211, heads_kv * (2 * group + 2), dim)), torch.float16)
        h = heads_kv * group
        q, k, v, at = wide[:, :h], wide[:, h:h + heads_kv], wide[:, h + heads_kv:h + 2 * heads_kv], wide[:, h + 2 * heads_kv:]
        o = torch.empty(211, h, dim, dtype=torch.float16, device="cuda")
        xp.xp_attn_prompt(q, k, v, cu, cu, 0.125, o)
        xp.xp_attn_prompt(q, k, v, cu, cu, 0.125, at)
        xp.xp_attn_prompt(q, k, v, cu, cu, 0.125, q)
        assert torch.equal(at, o) and torch.equal(q, o)
        for bad in (wide[:, 1:1 + h], wide[:, h - 1:2 * h - 1], wide[:, 2 * heads_kv:2 * heads_kv + h]):
            with pytest.raises(xp.XPError):
                xp.xp_attn_prompt(q, k, v, cu, cu, 0.125, bad)


@pytest.mark.parametrize("kv,group,dim,ty", [(2, 4, 128, "bf16"), (1, 2, 64, "f16"), (2, 2, 256, "bf16")])
def test_prompt_in_two_pieces_over_the_cache(kv, group, dim, ty):
    """The way of a prompt's later piece: both pieces' rows go into the cache as they come, the keys and values of
    all of it are read back, and the new rows attend to them; as tokens of a decode call they see the same."""
    rng = np.random.default_rng(dim)
    page, first, then = 64, [130, 0, 70], [45, 33, 1]
    rows, cols = [a + b for a, b in zip(first, then)], 3
    c = ref.Cache(kv, dim, page, 3 * cols, rng=rng)
    table = tables(rng, 3, cols, 3 * cols)
    d, buf, t = dims_of(c), on_device(c), dev(table)
    k, v = (dev(rng.normal(size=(sum(rows), kv, dim)), DT[ty]) for _ in "kv")
    q = dev(rng.normal(size=(sum(then), kv * group, dim)), DT[ty])
    cu, cu_q = ends(rows), ends(then)
    old = torch.from_numpy(np.concatenate([np.arange(cu[b], cu[b] + first[b]) for b in range(3)])).cuda()
    new = torch.from_numpy(np.concatenate([np.arange(cu[b] + first[b], cu[b + 1]) for b in range(3)])).cuda()
    xp.xp_kv_append(d, k[old], v[old], dev(ends(first)), ints([0, 0, 0]), t, buf)
    xp.xp_kv_append(d, k[new], v[new], dev(cu_q), ints(first), t, buf)
    kr, vr = torch.empty_like(k), torch.empty_like(v)
    xp.xp_kv_read(d, dev(cu), ints([0, 0, 0]), t, buf, kr, vr)
    out = torch.empty_like(q)
    xp.xp_attn_prompt(q, kr, vr, dev(cu_q), dev(cu), dim ** -0.5, out)
    check_prompt(q, kr, vr, cu_q, cu, out, dim ** -0.5)
    ref.append(c, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, [0, 0, 0], table)
    np.testing.assert_array_equal(buf.cpu().numpy(), c.b.reshape(-1))
    for b in range(3):                                     # the same rows as tokens of a decode call
        o = run_decode(c, buf, table[b:b + 1], np.array([rows[b]], dtype=np.int32), q[cu_q[b]:cu_q[b + 1]], dim ** -0.5,
                       q_rows=then[b])
        check_decode(c, table[b:b + 1], np.array([rows[b]]), q[cu_q[b]:cu_q[b + 1]], o, dim ** -0.5, 0, then[b])


def test_a_cache_of_more_than_4_gib():
    """Pages far apart in a large cache: the same calls over the same bytes in a small one give the same."""
    rng = np.random.default_rng(13)
    kv, dim, page, far = 2, 256, 1 << 15, 290                 # 17.8 MB a page: the last ones beyond 2^32 and 5e9 bytes
    small, large = xp.kv_dims(kv, dim, page, 4), xp.kv_dims(kv, dim, page, far)
    assert xp.xp_kv_bytes(large) > 5 * 10 ** 9
    ids = np.array([[240, 0], [289, 241]], dtype=np.int32)      # page 240 crosses 2^32
    one = xp.xp_kv_bytes(small) // 4
    assert 240 * one < 2 ** 32 < 241 * one
    n = [page + 700, page + 77]
    cu, cu1, start = ends(n), ends([1, 1]), [0, 0]
    k, v = (torch.randn(int(cu[-1]), kv, dim, device="cuda").to(torch.bfloat16) for _ in "kv")
    q = torch.randn(2, 8, dim, device="cuda").to(torch.bfloat16)
    w0 = torch.rand(2, kv, 2 * page, device="cuda")
    got = []
    for d, table in ((small, np.array([[0, 1], [2, 3]], dtype=np.int32)), (large, ids)):
        buf = torch.zeros(xp.xp_kv_bytes(d), dtype=torch.uint8, device="cuda")
        t, ln, w = dev(table), ints(n), w0.clone()
        xp.xp_kv_append(d, k, v, dev(cu), ints(start), t, buf)
        xp.xp_kv_append(d, k[:2], v[:2], dev(cu1), ints([n[0] - 1, n[1] - 1]), t, buf)   # the form for few rows
        ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, 8, 1, 2, max(n)), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        xp.xp_attn_decode(d, q, buf, t, ln, max(n), 0.06, out, ws, weights=w)
        kept = torch.empty(2, kv, page + 5, dtype=torch.int32, device="cuda")
        wk = w.clone()
        xp.xp_kv_evict(d, buf, t, ln, w, page + 5, t, kept, ln, w, sinks=4, recent=8)
        ko, vo = (torch.empty(2 * (page + 5), kv, dim, dtype=torch.float32, device="cuda") for _ in "kv")
        xp.xp_kv_read(d, dev(ends([page + 5] * 2)), ints(start), t, buf, ko, vo)
        k1, v1 = (torch.empty(2, kv, dim, dtype=torch.float32, device="cuda") for _ in "kv")
        xp.xp_kv_read(d, dev(cu1), ints([page + 4, page + 4]), t, buf, k1, v1)
        got.append((out, wk, w, kept, ln, ko, vo, k1, v1))
        del buf
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0] != 0).any() and (got[0][5] != 0).any() and torch.equal(got[0][7], got[0][5][[page + 4, 2 * page + 9]])


def test_bench_attention_cell():
    import bench
    r = bench.time_attn(2, 3, 1)
    assert set(r) == {"attention/%d" % n for n in bench.ATTN_ROWS} | {"attention/prompt"}
    b = bench.brief(r)
    assert all(v["layer_us"] > 0 for k, v in b.items() if k != "attention/prompt")
    assert b["attention/prompt"]["us"] > 0 and b["attention/prompt"]["tflops"] > 0
