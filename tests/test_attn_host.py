"""Host side of the 4-bit cache and attention entry points (no GPU): sizes, refusals
before any launch, and the tests' own reference against independent checks."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref
import attn_tiles as tiles

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1004)
BF16, F16, F32 = 0, 1, 2


def kd(kv=2, dim=64, page=64, pages=4):
    return ctypes.byref(xp.kv_dims(kv, dim, page, pages))


BAD_DIMS = [(0, 64, 64, 4), (1025, 64, 64, 4), (2, 32, 64, 4), (2, 96, 64, 4), (2, 512, 64, 4), (2, 64, 0, 4),
            (2, 64, 32, 4), (2, 64, 96, 4), (2, 64, -64, 4), (2, 64, 64, 0), (2, 64, 64, -1)]


def test_cache_bytes():
    # 4.25 bits a value, k and v
    for kv, dim, page, pages in ((8, 128, 256, 10), (1, 64, 64, 1), (3, 256, 192, 7)):
        assert xp.xp_kv_bytes(xp.kv_dims(kv, dim, page, pages)) * 8 == pages * page * kv * dim * 2 * 17 // 4
    for d in BAD_DIMS:
        assert xp.xp_kv_bytes(xp.kv_dims(*d)) == 0, d
    assert xp.lib().xp_kv_bytes(None) == 0


@pytest.mark.parametrize("d", BAD_DIMS)
def test_bad_cache_dims_refused(d):
    L, g = xp.lib(), ctypes.byref(xp.kv_dims(*d))
    assert L.xp_kv_append(g, 1, 1, 1, BF16, P, 1 << 20, P, 1 << 20, P, P, P, P, None) == xp.XP_ERR_SHAPE
    assert L.xp_kv_read(g, 1, 1, 1, BF16, P, P, P, P, P, 1 << 20, P, 1 << 20, None) == xp.XP_ERR_SHAPE
    assert L.xp_kv_evict(g, 1, 1, P, P, P, P, 1 << 20, 4, 0, 0, 1, P, P, P, P, 1 << 20, None) == xp.XP_ERR_SHAPE
    assert L.xp_attn_decode(g, 4, 1, 1, 1, 64, BF16, P, 1 << 20, 1.0, 0, P, P, P, P, 1 << 20, None, 0, P, 1 << 30,
                            None) == xp.XP_ERR_SHAPE
    assert L.xp_attn_decode_workspace_bytes(g, 4, 1, 1, 64) == 0


def _rows_call(name, **kw):
    a = dict(g=kd(), batch=1, cols=1, rows=3, ty=BF16, k=P, ks=128, v=P, vs=128, cu=P, start=P, table=P, cache=P)
    a.update(kw)
    L = xp.lib()
    if name == "xp_kv_append":
        return L.xp_kv_append(a["g"], a["batch"], a["cols"], a["rows"], a["ty"], a["k"], a["ks"], a["v"], a["vs"],
                              a["cu"], a["start"], a["table"], a["cache"], None)
    return L.xp_kv_read(a["g"], a["batch"], a["cols"], a["rows"], a["ty"], a["cu"], a["start"], a["table"], a["cache"],
                        a["k"], a["ks"], a["v"], a["vs"], None)


@pytest.mark.parametrize("name", ["xp_kv_append", "xp_kv_read"])
def test_row_calls_refuse(name):
    def call(**kw):
        return _rows_call(name, **kw)
    assert call(g=None) == xp.XP_ERR_NULL
    for key in ("k", "v", "cu", "start", "table", "cache"):
        assert call(**{key: None}) == xp.XP_ERR_NULL, key
    for kw in (dict(batch=-1), dict(batch=65536), dict(cols=0), dict(rows=-1), dict(ty=3), dict(ty=-1),
               dict(rows=1 << 29), dict(ks=120), dict(vs=64), dict(ks=132), dict(vs=129), dict(ty=F32, ks=130), dict(cols=1 << 26),
               dict(k=ODD), dict(v=ODD), dict(cache=ODD), dict(cu=ctypes.c_void_p(0x1002)),
               dict(table=ctypes.c_void_p(0x1001)), dict(start=ctypes.c_void_p(0x1002))):
        assert call(**kw) == xp.XP_ERR_SHAPE, kw
    none = dict(k=None, v=None, cu=None, start=None, table=None, cache=None)
    assert call(rows=0, **none) == xp.XP_OK
    assert call(batch=0, **none) == xp.XP_OK


@pytest.mark.parametrize("name", ["xp_kv_append", "xp_kv_read"])
def test_row_calls_refuse_launches_of_2_32_threads(name):
    """64 rows of a kv head are a workgroup of 256: 2^14 such blocks, the last one short, times 1,024 heads are one too many."""
    for rows in ((1 << 20) - 1, (1 << 20) - 63):
        assert _rows_call(name, g=kd(kv=1024), rows=rows, ks=65536, vs=65536) == xp.XP_ERR_SHAPE, rows


def _decode(**kw):
    a = dict(g=kd(), heads=4, q_rows=1, batch=1, cols=1, max_len=64, ty=BF16, q=P, qs=256, scale=1.0, window=0, cache=P,
             table=P, lens=P, out=P, os=256, weights=None, ws=0, work=P, bytes=1 << 30)
    a.update(kw)
    return xp.lib().xp_attn_decode(*[a[k] for k in ("g", "heads", "q_rows", "batch", "cols", "max_len", "ty", "q", "qs",
                                                     "scale", "window", "cache", "table", "lens", "out", "os", "weights",
                                                     "ws", "work", "bytes")], None)


def test_decode_refuses():
    assert _decode(g=None) == xp.XP_ERR_NULL
    for key in ("q", "cache", "table", "lens", "out", "work"):
        assert _decode(**{key: None}) == xp.XP_ERR_NULL, key
    inf, nan = float("inf"), float("nan")
    for kw in (dict(heads=0), dict(heads=3), dict(heads=65536), dict(q_rows=0), dict(q_rows=-1), dict(q_rows=65536),
               dict(batch=-1), dict(batch=65536), dict(cols=0), dict(max_len=-1), dict(ty=F32), dict(ty=7),
               dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan), dict(qs=248),
               dict(os=252), dict(qs=260), dict(os=258), dict(q=ODD), dict(out=ODD), dict(cache=ODD), dict(work=ODD),
               dict(lens=ctypes.c_void_p(0x1002)), dict(table=ctypes.c_void_p(0x1002)),
               dict(weights=P, ws=63), dict(weights=ctypes.c_void_p(0x1002), ws=64),
               dict(heads=65534, q_rows=65535, qs=1 << 30, os=1 << 30), dict(batch=65535, q_rows=4096)):
        assert _decode(**kw) == xp.XP_ERR_SHAPE, kw
    assert _decode(batch=0, q=None, cache=None, table=None, lens=None, out=None, work=None, bytes=0) == xp.XP_OK
    need = xp.xp_attn_decode_workspace_bytes(xp.kv_dims(2, 64, 64, 4), 4, 1, 1, 4096)
    assert need > 0
    assert _decode(max_len=4096, bytes=need - 1) == xp.XP_ERR_WORKSPACE


def test_evict_refuses():
    def call(**kw):
        a = dict(g=kd(), batch=1, cols=2, cache=P, table=P, lens=P, w=P, ws=128, keep=64, sinks=4, recent=8, dcols=1,
                 dst=P, kept=P, lo=P, wo=P, wos=64)
        a.update(kw)
        return xp.lib().xp_kv_evict(*[a[k] for k in ("g", "batch", "cols", "cache", "table", "lens", "w", "ws", "keep",
                                                     "sinks", "recent", "dcols", "dst", "kept", "lo", "wo", "wos")], None)
    assert call(g=None) == xp.XP_ERR_NULL
    for key in ("cache", "table", "lens", "w", "dst", "kept", "lo", "wo"):
        assert call(**{key: None}) == xp.XP_ERR_NULL, key
    W = ctypes.c_void_p(0x2000)
    for kw in (dict(batch=-1), dict(batch=65536), dict(cols=0), dict(dcols=0), dict(keep=0), dict(keep=-1),
               dict(keep=65), dict(sinks=-1), dict(recent=-1), dict(sinks=60, recent=5), dict(ws=127), dict(wos=63),
               dict(cache=ODD), dict(w=ctypes.c_void_p(0x1002)), dict(kept=ctypes.c_void_p(0x1002)),
               dict(w=W, wo=W, ws=128, wos=130), dict(sinks=0x7fffffff, recent=0x7fffffff)):
        assert call(**kw) == xp.XP_ERR_SHAPE, kw
    assert call(batch=0, cache=None, table=None, lens=None, w=None, dst=None, kept=None, lo=None, wo=None) == xp.XP_OK


def test_prompt_refuses():
    def call(**kw):
        a = dict(heads=4, kv=2, dim=64, batch=1, rq=5, rk=5, ty=BF16, q=P, qs=256, k=P, ks=128, v=P, vs=128, cq=P, ck=P,
                 scale=1.0, window=0, out=P, os=256)
        a.update(kw)
        return xp.lib().xp_attn_prompt(*[a[k] for k in ("heads", "kv", "dim", "batch", "rq", "rk", "ty", "q", "qs", "k", "ks",
                                                        "v", "vs", "cq", "ck", "scale", "window", "out", "os")], None)
    for key in ("q", "k", "v", "cq", "ck", "out"):
        assert call(**{key: None}) == xp.XP_ERR_NULL, key
    inf, nan = float("inf"), float("nan")
    for kw in (dict(heads=0), dict(kv=0), dict(heads=3), dict(kv=1025, heads=1025), dict(dim=32), dict(dim=96), dict(dim=0),
               dict(batch=-1), dict(batch=65536), dict(rq=-1), dict(rk=-1), dict(ty=F32), dict(ty=-1), dict(window=-1),
               dict(scale=0.0), dict(scale=-2.0), dict(scale=inf), dict(scale=nan), dict(qs=248), dict(ks=120), dict(vs=120),
               dict(os=248), dict(ks=1 << 24), dict(vs=1 << 24), dict(qs=258), dict(ks=132), dict(vs=130), dict(os=258), dict(q=ODD), dict(k=ODD), dict(v=ODD),
               dict(out=ODD), dict(cq=ctypes.c_void_p(0x1002)), dict(rq=1 << 28), dict(rq=0x7fffffff), dict(rk=0x7fffffff)):
        assert call(**kw) == xp.XP_ERR_SHAPE, kw
    assert call(rq=0, q=None, out=None) == xp.XP_OK
    assert call(batch=0, q=None, k=None, v=None, cq=None, ck=None, out=None) == xp.XP_OK


def test_binding_refuses_host_tensors():
    d = xp.kv_dims(2, 64, 64, 4)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        xp.xp_kv_append(d, x, x, i, i, i.view(1, 2), torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        xp.xp_attn_prompt(x, x, x, i, i, 1.0, x)
    with pytest.raises(ValueError):
        xp.xp_attn_prompt(x.float(), x, x, i, i, 1.0, x)


# ------------------------------------------------------- the tests' reference
def test_reference_tables_match_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.nan_to_num(t, nan=-1.0), np.nan_to_num(ref.E4M3, nan=-1.0))
    assert ref.SCALES[-1] == 448 and np.all(np.diff(ref.SCALES) > 0)


def test_reference_quantise_by_fractions():
    """Every code is a nearest multiple, ties to even; the scale is the smallest that reaches."""
    rng = np.random.default_rng(5)
    mags = [Fraction(m) for m in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]
    x = rng.normal(size=(40, 32)).astype(np.float32).astype(np.float64)
    x[1] *= 1e-3
    x[2] *= 900.0
    x[3] = np.round(x[3] * 4) / 4
    x[3, 0] = 6.0                                            # scale 1: quarters hit every midpoint
    x[4] = 0.0
    x[5, 0] = 6 * 448 * 1.01                                 # beyond the last scale
    x[6] *= 1e-6                                             # below the first scale's half step
    codes, byte = ref.quantise(x)
    for r in range(40):
        top = max(abs(Fraction(v)) for v in x[r])
        fit = [i for i in range(127) if 6 * Fraction(ref.SCALES[i]) >= top]
        assert byte[r, 0] == (fit[0] if fit else 126)
        s = Fraction(ref.SCALES[byte[r, 0]])
        for v, c in zip(x[r], codes[r]):
            if s == 0:
                assert c & 7 == 0
                continue
            dist = [abs(abs(Fraction(v)) - m * s) for m in mags]
            best = min(dist)
            near = [i for i in range(8) if dist[i] == best]
            assert (c & 7) in near and (len(near) == 1 or (c & 1) == 0), (r, v, c)


def test_reference_layout_is_a_bijection():
    """Every byte of a tile belongs to exactly one (position, pair of values) or (position, group)."""
    for dim in (64, 128, 256):
        c = ref.Cache(1, dim, 64, 1)
        seen = np.zeros(c.ng * 2176, dtype=int)
        for pos in range(64):
            for which in ("k", "v"):
                codes, odd, s = c.at(0, 0, pos, which)
                np.testing.assert_array_equal(codes[0::2], codes[1::2])
                seen[codes[0::2]] += 1
                seen[s] += 1
        assert (seen == 1).all()


def test_reference_attend_against_torch():
    rng = np.random.default_rng(9)
    q, k, v = (rng.normal(size=(n, 32)) for n in (6, 6, 6))
    out, p, _, _ = ref.attend(q, k, v, np.arange(6), 0.3)
    want = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in (q, k, v)), is_causal=True,
                                                            scale=0.3)[0].numpy()
    np.testing.assert_allclose(out, want, rtol=1e-12, atol=1e-14)
    out, p, _, _ = ref.attend(q, k, v, np.array([-1, 0, 5, 5, 5, 5]), 0.3, window=1)
    assert (out[0] == 0).all() and (p[0] == 0).all()
    np.testing.assert_allclose(out[1], v[0])
    np.testing.assert_allclose(out[2], v[5])


def test_evict_refuses_counts_that_its_steps_would_pass():
    """The kernels' steps of up to 8,192 positions stay below 2^31 for at most 2^31 - 8192 kept ones."""
    def call(keep):
        pages = (2 ** 31 - 1025) // 64
        return xp.lib().xp_kv_evict(kd(kv=1), 1, pages, P, P, P, P, 1 << 31, keep, 0, 0, pages, P, P, P, P, 1 << 31, None)
    for keep in (2 ** 31 - 8191, 2 ** 31 - 4096, 2 ** 31 - 1088):
        assert call(keep) == xp.XP_ERR_SHAPE, keep


def _share(a, sa, b, sb, rows, width):
    """Whether rows of `width` bytes at a, a + sa, ... and b, b + sb, ... share a byte."""
    return any(a + i * sa < b + j * sb + width and b + j * sb < a + i * sa + width for i in range(rows) for j in range(rows))


def test_decode_refuses_out_over_q():
    """Where rows meet, also rows of another stride; views that interleave without meeting pass (to the workspace
    check, which these calls fail)."""
    base, width = 1 << 20, 256
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(3000):
        rows = int(rng.integers(1, 6))
        qs, os_ = (int(rng.integers(32, 120)) * 8 for _ in "qo")
        if rng.random() < 0.5:
            os_ = qs
        out = base + 16 * int(rng.integers(-600, 600))
        for weights in (None, P):
            same = out == base and (os_ == qs or rows == 1)
            bad = (weights is not None or not same) and _share(base, 2 * qs, out, 2 * os_, rows, 2 * width)
            got = _decode(q_rows=rows, q=ctypes.c_void_p(base), qs=qs, out=ctypes.c_void_p(out), os=os_, weights=weights,
                          ws=64, bytes=0)
            assert got == (xp.XP_ERR_SHAPE if bad else xp.XP_ERR_WORKSPACE), (rows, qs, os_, out - base, weights)
            seen.add((bad, os_ == qs))
    assert len(seen) == 4
    at = ctypes.c_void_p(base)
    assert _decode(q_rows=3, q=at, out=at, bytes=0) == xp.XP_ERR_WORKSPACE
    assert _decode(q_rows=3, q=at, out=at, os=512, bytes=0) == xp.XP_ERR_SHAPE
    assert _decode(q_rows=3, q=at, out=at, weights=P, ws=64, bytes=0) == xp.XP_ERR_SHAPE
    far = 1 << 60
    assert _decode(q_rows=3, q=at, qs=far, out=ctypes.c_void_p(base + 16), os=far, bytes=0) == xp.XP_ERR_SHAPE
    assert _decode(q_rows=3, q=at, qs=far, out=ctypes.c_void_p(base + 512), os=far, bytes=0) == xp.XP_ERR_WORKSPACE


def test_other_calls_refuse_what_they_write_over_what_they_read():
    L, c = xp.lib(), ctypes.c_void_p
    at = 1 << 20

    def prompt(out, os_=256):
        return L.xp_attn_prompt(4, 2, 64, 1, 5, 5, BF16, c(at), 256, c(at + (1 << 16)), 128, c(at + (2 << 16)), 128, P, P, 1.0,
                                0, c(out), os_, None)
    for out in (at + 16, at - 512, at + 4 * 512 + 496, at + (1 << 16), at + (1 << 16) + 4 * 256 + 240, at + (2 << 16) - 2048):
        assert prompt(out) == xp.XP_ERR_SHAPE, out - at
    assert prompt(at, 512) == xp.XP_ERR_SHAPE

    def read(v, vs=128):
        return _rows_call("xp_kv_read", k=c(at), v=c(v), vs=vs)
    for v, vs in ((at, 128), (at + 16, 128), (at - 256 * 2, 128), (at - 256 * 2, 192)):
        assert read(v, vs) == xp.XP_ERR_SHAPE, v - at

    def evict(wo, wos=128):
        return L.xp_kv_evict(kd(), 2, 2, P, P, P, c(at), 128, 64, 0, 0, 1, P, P, P, c(wo), wos, None)
    for wo, wos in ((at + 4, 128), (at - 4 * 4 * 128 + 512, 128), (at + 512, 64), (at + 4 * 512 - 4, 128), (at, 256)):
        assert evict(wo, wos) == xp.XP_ERR_SHAPE, (wo - at, wos)


def test_decode_takes_2_22_units_at_any_length():
    """Units: blocks of 16 rows of a kv head, of 32 where it has more than 16 and head_dim is below 256."""
    for dim, heads, q_rows, batch in ((64, 1024, 1, 4096), (128, 1024, 16, 4096), (256, 1024, 16, 4096), (64, 1024, 32, 4096),
                                      (128, 2048, 16, 4096), (256, 1024, 32, 2048), (64, 1024, 33, 2048)):
        d = xp.kv_dims(1024, dim, 64, 4)
        for max_len in (0, 64, 20000, 1 << 30):
            assert xp.xp_attn_decode_workspace_bytes(d, heads, q_rows, batch, max_len) > 0, (dim, heads, q_rows, max_len)
            assert xp.xp_attn_decode_workspace_bytes(d, heads, q_rows, batch + 1, max_len) == 0, (dim, heads, q_rows, max_len)
            call = dict(g=ctypes.byref(d), heads=heads, q_rows=q_rows, max_len=max_len, qs=heads * dim, os=heads * dim,
                        out=ctypes.c_void_p(1 << 50), bytes=0)
            assert _decode(batch=batch, **call) == xp.XP_ERR_WORKSPACE
            assert _decode(batch=batch + 1, **call) == xp.XP_ERR_SHAPE


def test_prompt_takes_fewer_than_2_23_blocks():
    """Blocks of 64 rows of a kv head, rows_q * heads / kv_heads of them for each, and one more for each sequence."""
    def call(heads, kv, batch, rq):
        return xp.lib().xp_attn_prompt(heads, kv, 64, batch, rq, 5, BF16, None, 1 << 20, P, 1 << 20, P, 1 << 20, P, P, 1.0, 0,
                                       P, 1 << 20, None)
    for heads, kv, batch, rq in ((1024, 1024, 1, 64 * 8190), (2048, 1024, 1, 32 * 8190), (128, 128, 65535, 0),
                                 (1, 1, 1, 64 * (2 ** 23 - 2)), (129, 129, 60000, 64 * 5027)):
        blocks = (-(-rq * (heads // kv) // 64) + batch) * kv
        assert blocks + kv >= 1 << 23 > blocks
        assert call(heads, kv, batch, rq) == (xp.XP_ERR_NULL if rq else xp.XP_OK), (heads, kv, batch, rq)
        assert call(heads, kv, batch, rq + 64 * kv // heads) == xp.XP_ERR_SHAPE, (heads, kv, batch, rq)


@pytest.mark.parametrize("name", list(tiles.DECODE) + list(tiles.PROMPT))
def test_a_tile_left_out_or_doubled_is_told(name):
    """For the rows of the cases of attn_tiles (some of those where there are many), but for tiles of which a row
    sees fewer than eight positions."""
    if name in tiles.DECODE:
        case = tiles.DECODE[name]
        dim, window, places = case[2], case[5], sorted({p for _, _, p in tiles.decode_rows(case)})
    else:
        case = tiles.PROMPT[name]
        dim, window, places = case[2], case[5], [p for _, p in tiles.prompt_rows(case)]
    for place in places if len(places) <= 12 else places[::len(places) // 6]:
        c = tiles.counts(place, window)
        assert c.sum() == max(0, min(place + 1, window or place + 1))
        if np.count_nonzero(c) > 1:                        # one alone is all of the output, once or twice
            assert all(c[t] < 8 for t in tiles.not_told_apart(c, dim)), place


def test_the_tiles_form_of_attention():
    """Its closed form is the definition's: equal scores over values that name their tile."""
    for dim, at, window in ((64, 700, 0), (64, 5000, 0), (128, 400, 150)):
        n = at + 1
        col, val = tiles.column(np.arange(n) // 64, dim)
        v = np.zeros((n, dim))
        v[np.arange(n), col] = tiles.VALUES[val]
        out, _, _, _ = ref.attend(np.ones((1, dim)), np.ones((n, dim)), v, [at], 0.1, window)
        np.testing.assert_allclose(tiles.output(tiles.counts(at, window), dim), out[0], rtol=1e-12)
    codes = ref.E2M1[tiles.CODES]
    np.testing.assert_array_equal(codes, tiles.VALUES)
