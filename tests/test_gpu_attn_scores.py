"""GPU: attention where scores are far from the ordinary: finite queries and keys whose scores reach
far beyond fp16's range in log2 units."""
import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref
from test_gpu_attn import DT, dev, ends, filled, on_device, run_decode, tables

pytestmark = pytest.mark.gpu


def loud_cache(rng, kv, dim, page, pages):
    """K holds +-48 everywhere (code 7 or 15 times the scale 8), V values of ordinary size."""
    c = filled(rng, kv, dim, page, pages)
    n = c.ng * 1024
    c.b[..., :n] = 0x77 | (rng.integers(0, 2, c.b.shape[:3] + (n,)) * 0x80 + rng.integers(0, 2, c.b.shape[:3] + (n,)) * 0x08)
    c.b[..., n:n + c.ng * 64] = 0x50                       # E4M3 8.0
    return c


@pytest.mark.parametrize("ty,mag", [("f16", 32000.0), ("f16", 2000.0), ("bf16", 1e6), ("bf16", 1e30)])
@pytest.mark.parametrize("dim,group,q_rows,n", [(128, 4, 1, 300), (128, 8, 5, 300), (64, 8, 2, 5000), (256, 3, 1, 900)])
def test_decode_large_finite_scores(dim, group, q_rows, n, ty, mag):
    """Each row's query points along one key that it sees (of random signs, so that no other comes near):
    its weight is 1 to within 2^-1000 of it, every other's 0, and the output is that position's v, which the
    output type holds exactly. Scores reach mag * 48 * sqrt(dim) (2^19 .. 2^110 in log2 units)."""
    rng = np.random.default_rng(dim + n + int(np.log2(mag)))
    kv, page, batch = 2, 128, 3
    lens = np.array([n, 257, 70], dtype=np.int32)
    cols = -(-n // page)
    c = loud_cache(rng, kv, dim, page, batch * cols)
    table = tables(rng, batch, cols, batch * cols)
    q = np.zeros((batch * q_rows, kv * group, dim))
    want = np.zeros_like(q)
    for b in range(batch):
        for h in range(kv):
            k, _ = c.rows(table[b], h, int(lens[b]), "k")
            v, _ = c.rows(table[b], h, int(lens[b]), "v")
            for i in range(q_rows):
                for g in range(group):
                    j = int(rng.integers(0, lens[b] - q_rows + i + 1))
                    q[b * q_rows + i, h * group + g] = np.sign(k[j]) * mag * rng.uniform(1.0, 2.0)
                    want[b * q_rows + i, h * group + g] = v[j]
    out = run_decode(c, on_device(c), table, lens, dev(q, DT[ty]), dim ** -0.5, q_rows=q_rows)
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)


@pytest.mark.parametrize("ty", ["bf16", "f16"])
def test_decode_large_equal_scores(ty):
    """Two equal keys at the top of huge scores weigh a half each, wherever they lie (one wave, several, several
    pieces); v holds whole quarters there, so their mean is exact in both types."""
    rng = np.random.default_rng(9)
    kv, dim, page, n = 1, 64, 64, 6000
    cols = -(-n // page)
    c = loud_cache(rng, kv, dim, page, cols)
    table = tables(rng, 1, cols, cols)
    one = (np.full(dim, 6, dtype=np.uint8), np.full(2, 0x38, dtype=np.uint8))        # 4 in every column
    two = (np.full(dim, 12, dtype=np.uint8), np.full(2, 0x38, dtype=np.uint8))       # -2
    for at in ((5, 40), (6, 64 * 7 + 3), (100, 5990)):
        a, b = ((int(table[0, p // page]), 0, p % page) for p in at)
        c.put(*b, "k", *c.get(*a, "k"))
        c.put(*a, "v", *one)
        c.put(*b, "v", *two)
        k, _ = c.rows(table[0], 0, n, "k")
        q = dev(np.stack([np.sign(k[at[0]]) * m for m in rng.uniform(3e4, 6.5e4, 8)])[None], DT[ty])
        out = run_decode(c, on_device(c), table, np.array([n], dtype=np.int32), q, 0.125)
        assert (out == 1.0).all(), at


@pytest.mark.parametrize("ty,mag,key", [("f16", 32000.0, 1000.0), ("f16", 32000.0, 60000.0), ("bf16", 1e6, 1e6),
                                        ("bf16", 1e15, 1e18), ("f16", 100.0, 50.0)])
@pytest.mark.parametrize("kv,group,dim,nq,prefix", [(2, 4, 128, [300, 70], [0, 40]), (2, 2, 64, [200], [0]),
                                                    (1, 3, 256, [150], [130]), (64, 2, 64, [200, 130], [0, 70]),
                                                    (64, 2, 128, [200, 130], [0, 70])])
def test_prompt_large_finite_scores(kv, group, dim, nq, prefix, ty, mag, key):
    """As test_decode_large_finite_scores: scores reach mag * key * sqrt(dim) (2^16 .. 2^113 in log2 units), and
    each row's output is the v of the one key along which its query points. All forms of the kernel."""
    rng = np.random.default_rng(dim + kv + int(np.log2(mag * key)))
    nk = [a + b for a, b in zip(nq, prefix)]
    cu_q, cu_k = ends(nq), ends(nk)
    k = rng.choice([-key, key], size=(cu_k[-1], kv, dim))
    v = torch.from_numpy(rng.normal(size=k.shape)).to(DT[ty])
    q, want = np.zeros((cu_q[-1], kv * group, dim)), torch.zeros(int(cu_q[-1]), kv * group, dim, dtype=DT[ty])
    for b in range(len(nq)):
        for i in range(nq[b]):
            j = cu_k[b] + rng.integers(0, prefix[b] + i + 1, kv * group)
            heads = np.arange(kv * group) // group
            q[cu_q[b] + i] = np.sign(k[j, heads]) * mag * rng.uniform(1.0, 2.0, (kv * group, 1))
            want[cu_q[b] + i] = v[torch.from_numpy(j), torch.from_numpy(heads)]
    q, k, v = dev(q, DT[ty]), dev(k, DT[ty]), v.cuda()
    out = torch.empty_like(q)
    xp.xp_attn_prompt(q, k, v, dev(cu_q), dev(cu_k), dim ** -0.5, out)
    np.testing.assert_array_equal(out.cpu().double().numpy(), want.double().numpy())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ty", ["bf16", "f16"])
def test_prompt_large_equal_scores(dim, ty):
    """Two equal keys at the top of huge scores, in one tile and in different ones, weigh a half each."""
    rng = np.random.default_rng(dim)
    n = 400
    k = rng.choice([-1000.0, 1000.0], size=(n, 1, dim))
    v = rng.normal(size=(n, 1, dim))
    pairs = [(0, 1), (3, 60), (10, 200), (130, 390)]
    for a, b in pairs:
        k[b], v[a], v[b] = k[a], 4.0, -2.0
    q = rng.choice([-1.0, 1.0], size=(n, 4, dim))
    for h, (a, b) in enumerate(pairs):
        q[b:, h] = np.sign(k[a, 0]) * rng.uniform(3e4, 6.5e4, (n - b, 1))
    out = torch.empty(n, 4, dim, dtype=DT[ty], device="cuda")
    cu = dev(ends([n]))
    xp.xp_attn_prompt(dev(q, DT[ty]), dev(k, DT[ty]), dev(v, DT[ty]), cu, cu, dim ** -0.5, out)
    for h, (a, b) in enumerate(pairs):
        assert (out[b:, h] == 1.0).all(), h


@pytest.mark.parametrize("nats,spread", [(16.3, 0.0), (17.5, 0.0), (17.5, 3.0)])
@pytest.mark.parametrize("kv,group,dim,n", [(1, 2, 64, 8192), (1, 2, 128, 8192), (1, 1, 256, 4096), (64, 2, 64, 2048),
                                            (64, 2, 128, 2048)])
def test_prompt_f16_long_tail_of_small_weights(kv, group, dim, n, nats, spread):
    """One key that stands out, with a value of 0, and many that weigh e^-16 to e^-19 of it each: the output is
    what these add up to.

    Scores are one product each, exact in fp32. The bound, relative to the output (all terms are positive): half a
    step of the output, a rounding of each weight in the products and in the sum, 2^-11 each; fp32 sums of n terms
    and the exponential, n 2^-24 + 2^-19; weights below fp16's normal numbers, held as 2^13 times p or more,
    are off by 2^-38 in the products and in the sum, against their mean."""
    rng = np.random.default_rng(n + kv)
    rows = 130
    k = np.zeros((n, kv, dim))
    k[1:, :, 0] = -nats + spread * (rng.random((n - 1, kv)) - 0.5)
    v = rng.uniform(8.0, 24.0, size=(n, kv, dim))
    v[0] = 0.0
    q = np.zeros((rows, kv * group, dim))
    q[:, :, 0] = 1.0
    q, k, v = (dev(x, torch.float16) for x in (q, k, v))
    out = torch.empty_like(q)
    xp.xp_attn_prompt(q, k, v, dev(ends([rows])), dev(ends([n])), 1.0, out)
    e = torch.exp(k[:, :, 0].double())                                  # [n][kv]
    num, den = torch.cumsum(e[:, :, None] * v.double(), 0), torch.cumsum(e, 0)
    want = (num / den[:, :, None])[n - rows:].repeat_interleave(group, 1)
    assert float(want.min()) > 2.0 ** -13
    rel = 3 * 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -19 + 2 * 2.0 ** -38 / float(e[1:].mean())
    worst = float(((out.double() - want).abs() / want).max())
    print("relative error %.2e of %.2e" % (worst, rel), flush=True)
    assert worst <= rel


@pytest.mark.parametrize("dim,group,q_rows,n", [(128, 1, 1, 300), (64, 8, 3, 5000), (256, 2, 1, 700)])
@pytest.mark.parametrize("offset", [300.0, 3e3, 3e4, 3e5])
def test_decode_weights_add_up_at_large_scores(offset, dim, group, q_rows, n):
    """Scores of a few units of spread around a large offset (in log2 units): what a row adds to the weights is a
    probability distribution, whatever the scores' size.

    Both kernels form the same scores and take the same exponentials of their differences: two exponentials and
    their arguments' roundings, 2^-20 in all; a lane's share of the sum is at most n / 4 fp32 adds, the rows' sum
    at a position q_rows * group more."""
    rng = np.random.default_rng(int(offset) + dim)
    kv, page = 2, 64
    cols = -(-n // page)
    c = filled(rng, kv, dim, page, cols)
    c.b[..., :1024] = 0x77                                 # group 0 of every key: 48 everywhere
    c.b[..., c.ng * 1024:c.ng * 1024 + 64] = 0x50
    table = tables(rng, 1, cols, cols)
    q = rng.normal(size=(q_rows, kv * group, dim))
    scale = 0.5 * dim ** -0.5
    q[:, :, :32] = offset / (np.log2(np.e) * scale * 48.0 * 32.0) * rng.uniform(1.0, 1.2, (q_rows, kv * group, 1))
    w = torch.zeros(1, kv, cols * page, device="cuda")
    run_decode(c, on_device(c), table, np.array([n], dtype=np.int32), dev(q, torch.bfloat16), scale, q_rows=q_rows, weights=w)
    total = w.double().sum(-1).cpu().numpy() / (q_rows * group)
    bound = 2.0 ** -20 + (n / 4 + q_rows * group) * 2.0 ** -24
    print("off by %.1e of %.1e" % (np.abs(total - 1).max(), bound), flush=True)
    assert (np.abs(total - 1) <= bound).all(), total


@pytest.mark.parametrize("ty,mag", [("f16", 32000.0), ("bf16", 1e6), ("bf16", 1e30)])
def test_decode_weights_of_large_finite_scores(ty, mag):
    """As test_decode_large_finite_scores: each row adds 1 at the position along which its query points."""
    rng = np.random.default_rng(7)
    kv, group, dim, page, n, q_rows = 2, 4, 128, 64, 4500, 2
    cols = -(-n // page)
    c = loud_cache(rng, kv, dim, page, cols)
    table = tables(rng, 1, cols, cols)
    q, want = np.zeros((q_rows, kv * group, dim)), np.zeros((1, kv, cols * page))
    for h in range(kv):
        k, _ = c.rows(table[0], h, n, "k")
        for i in range(q_rows):
            for g in range(group):
                j = int(rng.integers(0, n - 1))
                q[i, h * group + g] = np.sign(k[j]) * mag * rng.uniform(1.0, 2.0)
                want[0, h, j] += 1.0
    w = torch.zeros(1, kv, cols * page, device="cuda")
    run_decode(c, on_device(c), table, np.array([n], dtype=np.int32), dev(q, DT[ty]), dim ** -0.5, q_rows=q_rows, weights=w)
    np.testing.assert_array_equal(w.cpu().numpy(), want)


def test_decode_a_sequence_of_2_30_positions_among_short_ones():
    """The longest sequence of a batch that is worked on in order of length, of 2^24 tiles: a float no longer tells
    its tiles from its tiles and one. All values are 1 and all scores equal, so every output is 1 exactly. Pages
    that are only read may be shared: one page of 2^20 positions stands for all. max_len is smaller than the
    longest length, as a launch may be, so nothing is cut."""
    kv, page, batch, tile = 5, 1 << 20, 64, 2 * 2176
    d = xp.kv_dims(kv, 64, page, 1)
    one = torch.zeros(tile, dtype=torch.uint8)
    one[2048:2176] = 0x38                                  # K: zeros
    one[2176:2176 + 2048] = 0x22                           # V: ones
    one[2176 + 2048:] = 0x38
    buf = one.cuda().repeat(kv * (page // 64))
    assert buf.numel() == xp.xp_kv_bytes(d)
    table = torch.zeros(batch, 1 << 10, dtype=torch.int32, device="cuda")
    lens = torch.arange(1, batch + 1, dtype=torch.int32, device="cuda")
    lens[17] = 1 << 30
    q = torch.randn(batch, kv, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, kv, 1, batch, 1024), dtype=torch.uint8, device="cuda")
    xp.xp_attn_decode(d, q, buf, table, lens, 1024, 0.125, out, ws)
    assert (out == 1.0).all(), (out != 1.0).any(-1).nonzero().tolist()


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("kv,group,dim", [(1, 2, 64), (1, 2, 128), (1, 1, 256), (64, 2, 64), (64, 2, 128)])
@pytest.mark.parametrize("climb", [0.6, 1.9, 2.1, 7.8, 8.2, 30.0, -3.0])
def test_prompt_scores_that_climb_from_tile_to_tile(climb, kv, group, dim, ty):
    """By less and by more than the running maximum may lag behind, in powers of two a tile, over 20 tiles: it is
    raised never, now and then, or at every tile.

    Scores are one product each. The bound: half a step of the output; a rounding of each weight in the products and
    in the sum; fp16 weights below its normal numbers, 2^-38 of the largest each, in both; fp32 sums of n terms, the
    maximum's product with the factor and the exponential, n 2^-24 + 2^-16 + 2^-19."""
    rng = np.random.default_rng(dim + kv)
    n, rows = 1290, 150
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[ty]
    k = np.zeros((n, kv, dim))
    k[:, :, 0] = climb * (np.arange(n) // 64)[:, None] + rng.uniform(-0.5, 0.5, (n, kv))
    v = rng.normal(size=k.shape)
    q = np.zeros((rows, kv * group, dim))
    q[:, :, 0] = 1.0
    q, k, v = (dev(x, DT[ty]) for x in (q, k, v))
    out = torch.empty_like(q)
    xp.xp_attn_prompt(q, k, v, dev(ends([rows])), dev(ends([n])), float(np.log(2.0)), out)
    kd, vd, got = k.double().cpu().numpy(), v.double().cpu().numpy(), out.double().cpu().numpy()
    worst = 0.0
    for h in sorted({0, kv // 2, kv - 1}):
        s = np.where(np.arange(n)[None, :] <= np.arange(n - rows, n)[:, None], kd[:, h, 0] * np.log(2.0), -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        p = e / e.sum(1, keepdims=True)
        want, wide = p @ vd[:, h], p @ np.abs(vd[:, h])
        tol = half * np.abs(want) + (half + n * 2.0 ** -24 + 2.0 ** -16 + 2.0 ** -19) * (wide + np.abs(want))
        tol += (2.0 ** -38 if ty == "f16" else 0.0) * (np.abs(vd[:, h]).sum(0) + n * np.abs(want)) + 1e-30
        for g in range(group):
            err = np.abs(got[:, h * group + g] - want)
            assert (err <= tol).all(), (h, g, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
    print("share of the bound: %.2f" % worst, flush=True)
