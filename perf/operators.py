"""Cases that time attention over a 4-bit key/value cache, the cache's own operators and attention over a whole prompt.

Each case is one call (or the two calls that belong together) with data as a
serving program holds it: rows of q, k and v in 16 or 32 bits, a paged cache of
e2m1 codes with one E4M3 scale per 32 values, page tables and lengths on the
GPU. The plain form is elementary torch arithmetic in fp32 on the same bytes;
``exact`` is the definition in float64, written apart from it.

Cache layout (one tile = 64 positions of one kv head; a page holds page / 64
tiles for each kv head, [kv_heads][page / 64][tile]); NG = head_dim / 32:
  K codes   16-byte chunk (pos, g)  at g * 1024 + pos * 16, low nibble = even k;
  K scales  byte (pos, g)           at NG * 1024 + g * 64 + (pos % 16) * 4 + pos / 16;
  V codes   8-byte chunk (pos, h)   at NG * 1088 + h * 512 + pos * 8, h = 16 values each;
  V scales  byte (pos, g)           at NG * 2112 + g * 64 + (pos / 4 % 4) * 16 + (pos / 16) * 4 + pos % 4.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 32 sequences: each appends its token's k and v; read back
        {"name": "append_step", "op": "append", "batch": 32, "kv_heads": 8, "dim": 128, "page": 64, "len": 2000,
         "rows": 1, "type": "bf16"},
        # six prompts of different lengths enter the cache, straight from fp32 projections; read back
        {"name": "append_prompts", "op": "append", "batch": 6, "kv_heads": 8, "dim": 128, "page": 256, "len": 0,
         "rows": 2047, "type": "f32"},
        # the shortest call: one sequence, a short context, where only latency counts
        {"name": "decode_short", "op": "decode", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "len": 300, "q_rows": 1, "window": 0, "weights": False, "idle": 0, "type": "bf16"},
        # a full serving batch of ragged contexts, two of its slots idle
        {"name": "decode_batch", "op": "decode", "batch": 64, "heads": 64, "kv_heads": 8, "dim": 128, "page": 256,
         "len": 8192, "q_rows": 1, "window": 0, "weights": False, "idle": 2, "type": "bf16"},
        # one very long document, few kv heads
        {"name": "decode_long", "op": "decode", "batch": 1, "heads": 32, "kv_heads": 4, "dim": 128, "page": 256,
         "len": 131072, "q_rows": 1, "window": 0, "weights": False, "idle": 0, "type": "f16"},
        # four drafted tokens a sequence, every head its own cache, a sliding window
        {"name": "decode_drafted_window", "op": "decode", "batch": 8, "heads": 16, "kv_heads": 16, "dim": 64,
         "page": 128, "len": 6001, "q_rows": 4, "window": 1500, "weights": False, "idle": 0, "type": "f16"},
        # a step that also adds each position's attention weight to what an eviction goes by
        {"name": "decode_weights", "op": "decode", "batch": 8, "heads": 32, "kv_heads": 8, "dim": 128, "page": 256,
         "len": 16384, "q_rows": 1, "window": 0, "weights": True, "idle": 0, "type": "bf16"},
        # a short question on its own
        {"name": "prompt_short", "op": "prompt", "batch": 1, "heads": 16, "kv_heads": 16, "dim": 64, "len": 77,
         "prefix": 0, "window": 0, "type": "f16"},
        # eight prompts of different lengths, packed into one call
        {"name": "prompt_packed", "op": "prompt", "batch": 8, "heads": 32, "kv_heads": 8, "dim": 128, "len": 1000,
         "prefix": 0, "window": 0, "type": "bf16"},
        # one long document
        {"name": "prompt_long", "op": "prompt", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "len": 8192,
         "prefix": 0, "window": 0, "type": "bf16"},
        # one sequence past its budget by a little
        {"name": "evict_one", "op": "evict", "batch": 1, "kv_heads": 8, "dim": 128, "page": 64, "len": 1100,
         "keep": 1024, "sinks": 4, "recent": 64},
        # a batch of long contexts cut to a quarter
        {"name": "evict_batch", "op": "evict", "batch": 8, "kv_heads": 8, "dim": 128, "page": 256, "len": 16384,
         "keep": 4096, "sinks": 4, "recent": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "decode", "prompt", "prompt", "evict"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 8, 16])
    page = rng.choice([64, 128, 192, 256])
    if op == "append":
        batch = _log(rng, 1, 64)
        return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "page": page, "len": rng.randint(0, 3000),
                "rows": _log(rng, 1, max(1, 12000 // batch)), "type": rng.choice(["bf16", "f16", "f32"])}
    if op == "decode":
        batch = _log(rng, 1, 64)
        room = 64 * 8192 * 8 * 128 // (batch * kv * dim)
        return {"op": op, "batch": batch, "heads": kv * rng.choice([1, 2, 4, 5, 8]), "kv_heads": kv, "dim": dim,
                "page": page, "len": _log(rng, 17, min(131072, room)), "q_rows": rng.choice([1, 1, 1, 2, 5]),
                "window": rng.choice([0, 0, 0, 700]), "weights": rng.random() < 0.3,
                "idle": 1 if batch > 4 and rng.random() < 0.5 else 0, "type": rng.choice(["bf16", "f16"])}
    if op == "prompt":
        batch = _log(rng, 1, 16)
        heads = kv * rng.choice([1, 2, 4])
        room = int(math.sqrt(8192 * 8192 * 32 * 128 / (batch * heads * dim)))
        n = _log(rng, 16, min(8192, room))
        return {"op": op, "batch": batch, "heads": heads, "kv_heads": kv, "dim": dim, "len": n,
                "prefix": rng.choice([0, 0, n // 3]), "window": rng.choice([0, 0, 0, 500]),
                "type": rng.choice(["bf16", "f16"])}
    batch = _log(rng, 1, 8)
    n = _log(rng, 200, 16384)
    return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "page": page, "len": n,
            "keep": max(96, int(n * rng.uniform(0.2, 0.95))), "sinks": rng.choice([0, 4]),
            "recent": rng.choice([16, 64])}


def _spread(batch, most, least=1):
    """Lengths of a ragged batch: the first is the longest, the others lie anywhere from an eighth of it up."""
    return [max(least, int(most * (1.0 - 0.875 * ((0.618034 * b) % 1.0)))) for b in range(batch)]


def _lens(case):
    """(cached positions, new rows) of each sequence."""
    b, n = case["batch"], case["len"]
    if case["op"] == "append":
        return _spread(b, n, 0), ([1] * b if case["rows"] == 1 else _spread(b, case["rows"]))
    if case["op"] == "prompt":
        rows = _spread(b, n)
        return [min(case["prefix"], 2 * r) for r in rows], rows
    lens = _spread(b, n, case.get("q_rows", 1))
    for i in range(case.get("idle", 0)):
        lens[-1 - 3 * i] = 0
    return lens, [case.get("q_rows", 1)] * b


# ----------------------------------------------------------------- inputs
def _table(g, batch, columns, page_count):
    """A page table whose pages lie anywhere in the pool; the unused rest of the pool follows."""
    order = torch.randperm(page_count, generator=g, device="cuda").to(torch.int32)
    return order[:batch * columns].view(batch, columns), order[batch * columns:]


def _cache(g, pages, kv_heads, dim, page):
    """A filled cache: codes as quantised normal values have them, scales from 0.2 to 0.6."""
    ng = dim // 32
    normal = torch.tensor([-1.86, -1.32, -1.01, -0.78, -0.58, -0.40, -0.24, -0.08], device="cuda") / 0.37
    near = (normal.abs()[:, None] > torch.tensor(MIDS, device="cuda")).sum(1)
    codes = torch.cat([near + 8, near]).to(torch.uint8)
    pair = (codes[:, None] + 16 * codes[None, :]).view(-1)
    tiles = pages * kv_heads * (page // 64)
    cache = torch.randint(0, 256, (tiles, ng * 2176), generator=g, device="cuda", dtype=torch.uint8)
    cache = pair[cache.int()]
    for at in (ng * 1024, ng * 2112):
        cache[:, at:at + ng * 64] = torch.randint(0x25, 0x32, (tiles, ng * 64), generator=g, device="cuda",
                                                  dtype=torch.uint8)
    return cache.view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)
    cached, rows = _lens(c)
    batch, kv, dim = c["batch"], c["kv_heads"], c["dim"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    ends = lambda v: ints(np.concatenate([[0], np.cumsum(v)]).tolist())  # noqa: E731
    s = {"case": c, "batch": batch, "kv": kv, "dim": dim, "scale": 1.0 / math.sqrt(dim)}
    if c["op"] == "prompt":
        dt = TYPES[c["type"]]
        keys = [p + r for p, r in zip(cached, rows)]
        s["q"] = (2.0 * normal(sum(rows), c["heads"], dim)).to(dt)
        s["k"], s["v"] = normal(sum(keys), kv, dim).to(dt), normal(sum(keys), kv, dim).to(dt)
        s["cu_q"], s["cu_k"] = ends(rows), ends(keys)
        s["max_q"], s["max_k"] = max(rows), max(keys)
        s["out"] = torch.empty_like(s["q"])
        return s
    page = c["page"]
    most = max(n + r for n, r in zip(cached, rows)) if c["op"] == "append" else max(cached)
    columns = -(-most // page)
    s["columns"], s["page"], s["max_len"] = columns, page, most
    if c["op"] == "append":
        pages = batch * columns + 3
        s["table"], _ = _table(g, batch, columns, pages)
        s["pages"], dt = pages, TYPES[c["type"]]
        total = sum(rows)
        # k has a few channels that are much larger than the rest, as keys do
        loud = 1.0 + 7.0 * (torch.rand(kv, dim, generator=g, device="cuda") < 0.03).float()
        s["k"], s["v"] = (normal(total, kv, dim) * loud).to(dt), normal(total, kv, dim).to(dt)
        s["cu"], s["start"], s["rows"] = ends(rows), ints(cached), total
        s["cache"] = torch.zeros(pages * kv * page // 64 * (dim // 32) * 2176, dtype=torch.uint8, device="cuda")
        s["k_out"] = torch.empty(total, kv, dim, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["lens"] = ints(cached)
    if c["op"] == "decode":
        pages, dt = batch * columns + 3, TYPES[c["type"]]
        s["table"], _ = _table(g, batch, columns, pages)
        s["pages"] = pages
        s["cache"] = _cache(g, pages, kv, dim, page)
        s["q"] = (2.0 * normal(batch * c["q_rows"], c["heads"], dim)).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["weights"] = 0.1 * torch.rand(batch, kv, columns * page, generator=g, device="cuda") if c["weights"] else None
        return s
    kept = -(-c["keep"] // page)
    pages = batch * (columns + kept) + 3
    s["table"], rest = _table(g, batch, columns, pages)
    s["dst"], s["pages"] = rest[:batch * kept].view(batch, kept), pages
    s["dst_columns"] = kept
    s["cache"] = _cache(g, pages, kv, dim, page)
    # accumulated weights fall off steeply; positions that no step has weighed yet hold zero
    w = torch.rand(batch, kv, columns * page, generator=g, device="cuda")
    s["weights"] = torch.where(w < 0.1, torch.zeros_like(w), w ** 6)
    s["weights_out"] = torch.zeros(batch, kv, kept * page, device="cuda")
    s["kept"] = torch.empty(batch, kv, c["keep"], dtype=torch.int32, device="cuda")
    s["lens_out"] = torch.empty(batch, dtype=torch.int32, device="cuda")
    s["cu"] = ends([min(n, c["keep"]) for n in cached])
    s["start"], s["rows"] = torch.zeros_like(s["lens"]), sum(min(n, c["keep"]) for n in cached)
    s["k_out"] = torch.empty(s["rows"], kv, dim, dtype=torch.bfloat16, device="cuda")
    s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ------------------------------------------------------ the framework's calls
def _own(s):
    from fp4_routed_expert_xp_amd import xp
    c = s["case"]
    if c["op"] == "prompt":
        xp.xp_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["scale"], s["out"], window=c["window"])
        return s["out"]
    kd = xp.kv_dims(s["kv"], s["dim"], s["page"], s["pages"])
    if c["op"] == "append":
        xp.xp_kv_append(kd, s["k"], s["v"], s["cu"], s["start"], s["table"], s["cache"])
        xp.xp_kv_read(kd, s["cu"], s["start"], s["table"], s["cache"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if c["op"] == "decode":
        if "ws" not in s:
            s["ws"] = torch.empty(xp.xp_attn_decode_workspace_bytes(kd, c["heads"], c["q_rows"], s["batch"],
                                                                    s["max_len"]), dtype=torch.uint8, device="cuda")
        xp.xp_attn_decode(kd, s["q"], s["cache"], s["table"], s["lens"], s["max_len"], s["scale"], s["out"], s["ws"],
                          q_rows=c["q_rows"], window=c["window"], weights=s["weights"])
        return (s["out"], s["weights"]) if c["weights"] else s["out"]
    xp.xp_kv_evict(kd, s["cache"], s["table"], s["lens"], s["weights"], c["keep"], s["dst"], s["kept"], s["lens_out"],
                   s["weights_out"], sinks=c["sinks"], recent=c["recent"])
    xp.xp_kv_read(kd, s["cu"], s["start"], s["dst"], s["cache"], s["k_out"], s["v_out"])
    return s["kept"], s["lens_out"], s["weights_out"], s["k_out"], s["v_out"]


# ------------------------------------------------------------- plain forms
def _values(codes):
    """Code bytes [..., n] to the 2n values they stand for, without their scale."""
    lut = torch.tensor(E2M1, device=codes.device)
    return lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]


def _e4m3(b):
    return b.contiguous().view(torch.float8_e4m3fn).float()


def _cached(s, table):
    """K and V [batch][kv][position][dim] of all positions of the table's pages, fp32."""
    ng, kv, n64 = s["dim"] // 32, s["kv"], s["page"] // 64
    t = s["cache"].view(s["pages"], kv, n64, ng * 2176)[table.int()].transpose(1, 2).flatten(2, 3)  # [B][kv][tile][bytes]
    kc = _values(t[..., :ng * 1024].unflatten(-1, (ng, 64, 16)))
    ks = _e4m3(t[..., ng * 1024:ng * 1088]).unflatten(-1, (ng, 16, 4)).transpose(-1, -2).flatten(-2)
    k = (kc * ks[..., None]).transpose(-3, -2).flatten(-2).flatten(2, 3)
    vc = _values(t[..., ng * 1088:ng * 2112].unflatten(-1, (2 * ng, 64, 8)))
    vs = _e4m3(t[..., ng * 2112:]).unflatten(-1, (ng, 4, 4, 4)).transpose(-3, -2).flatten(-3)
    v = (vc.unflatten(-3, (ng, 2)) * vs[..., None, :, None]).flatten(-4, -3).transpose(-3, -2).flatten(-2)
    return k, v.flatten(2, 3)


def _softmax(x, see):
    """Probabilities over the last axis among what `see` shows; rows that see nothing get zeros."""
    x = x.masked_fill_(~see, float("-inf"))
    e = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


def _visible(q_pos, k_pos, window):
    see = k_pos <= q_pos
    return see & (k_pos > q_pos - window) if window else see


def _decode(s):
    c, b, kv, dim, nq = s["case"], s["batch"], s["kv"], s["dim"], s["case"]["q_rows"]
    group = c["heads"] // kv
    k, v = _cached(s, s["table"])
    n = k.shape[2]
    q = s["q"].float().view(b, nq, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(b, kv, nq * group, dim)
    x = torch.matmul(q * s["scale"], k.transpose(-1, -2).contiguous())
    q_pos = (s["lens"][:, None] - nq + torch.arange(nq, device="cuda")).repeat_interleave(group, 1)[:, None, :, None]
    p = _softmax(x, _visible(q_pos, torch.arange(n, device="cuda"), c["window"]))
    o = torch.matmul(p, v).view(b, kv, nq, group, dim).permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["q"].dtype)
    if not c["weights"]:
        return o
    s["weights"] += p.sum(2)
    return o, s["weights"]


def _prompt(s):
    c, b, kv = s["case"], s["batch"], s["kv"]
    lq, lk = s["cu_q"].diff(), s["cu_k"].diff()
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    row_q = (s["cu_q"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    row_k = (s["cu_k"][:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"].float()[row_q].unflatten(2, (kv, -1)).permute(0, 2, 3, 1, 4)                 # [B][kv][group][i][dim]
    k, v = (s[n].float()[row_k].permute(0, 2, 1, 3)[:, :, None] for n in ("k", "v"))      # [B][kv][1][j][dim]
    x = torch.matmul(q * s["scale"], k.transpose(-1, -2).contiguous())
    q_pos = (lk - lq)[:, None, None] + i[:, None]
    see = _visible(q_pos, j, c["window"]) & (j < lk[:, None, None])
    o = torch.matmul(_softmax(x, see[:, None, None]), v).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B][i][heads][dim]
    at = torch.arange(s["q"].shape[0], device="cuda")
    of = torch.searchsorted(s["cu_q"], at, right=True) - 1
    return o[of, at - s["cu_q"][of]].to(s["q"].dtype)


def _quantised(x):
    """The values that the cache holds for x [rows][kv][dim]: in groups of 32 the smallest E4M3 scale of which six
    reach the largest magnitude, and the nearest e2m1 multiple of it (ties to the even code)."""
    x = x.float().unflatten(-1, (-1, 32))
    scales = _e4m3(torch.arange(0, 127, device="cuda", dtype=torch.uint8))
    s = scales[torch.searchsorted(6.0 * scales, x.abs().amax(-1)).clamp(max=126)][..., None]
    a = x.abs()
    up = [a > m * s if n % 2 == 0 else a >= m * s for n, m in enumerate(MIDS)]
    code = torch.stack(up).sum(0)
    lut = torch.tensor(E2M1[:8], device="cuda")
    return (torch.where(s > 0, lut[code], torch.zeros_like(a)) * s * torch.sign(x)).flatten(-2)


def _evict(s):
    c, b, kv, keep = s["case"], s["batch"], s["kv"], s["case"]["keep"]
    n, lens = s["weights"].shape[-1], s["lens"][:, None, None]
    at = torch.arange(n, device="cuda")
    held = (at < c["sinks"]) | (at >= lens - c["recent"])
    w = torch.where(held, torch.full_like(s["weights"], float("inf")), s["weights"]).masked_fill(at >= lens, -1.0)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    rank = torch.arange(keep, device="cuda")
    kept = torch.sort(torch.where(rank < lens, best, torch.full_like(best, n)), dim=-1).values
    there = kept < n
    src = kept.clamp(max=n - 1)
    new = torch.zeros_like(s["weights_out"])
    new[..., :keep] = torch.where(there, torch.gather(s["weights"], 2, src), torch.zeros_like(new[..., :keep]))
    row = torch.arange(s["rows"], device="cuda")
    of = torch.searchsorted(s["cu"], row, right=True) - 1
    src = src[of, :, row - s["cu"][of]]                                                    # [row][kv]
    head = torch.arange(kv, device="cuda")
    k, v = (t[of[:, None], head, src].to(torch.bfloat16) for t in _cached(s, s["table"]))
    return (torch.where(there, kept, torch.full_like(kept, -1)).int(), s["lens"].clamp(max=keep), new, k, v)


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "append":
        return _quantised(s["k"]).to(torch.bfloat16), _quantised(s["v"]).to(torch.bfloat16)
    return {"decode": _decode, "prompt": _prompt, "evict": _evict}[op](s)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    cached, rows = _lens(c)
    kv, dim = c["kv_heads"], c["dim"]
    held = kv * dim * 17 // 16          # bytes of one cached position: k and v, 4.25 bits a value
    if c["op"] == "append":
        width = 4 if c["type"] == "f32" else 2
        # rows in, codes and scales out, then in again, and the values out
        return {"bytes": sum(rows) * (2 * kv * dim * width + 2 * held + 2 * kv * dim * 2), "flops": 0}
    if c["op"] == "evict":
        kept = [min(n, c["keep"]) for n in cached]
        # the weights in, the kept positions in and out, then in again and their values out
        return {"bytes": sum(cached) * kv * 4 + sum(kept) * (3 * held + kv * 8 + 2 * kv * dim * 2), "flops": 0}
    keys = [n if c["op"] == "decode" else n + r for n, r in zip(cached, rows)]
    seen = touched = 0
    for n, r in zip(keys, rows):
        if not n:
            continue
        first = n - r                                  # position of the sequence's first query
        p = np.arange(first, n, dtype=np.int64)
        low = np.maximum(0, p - c["window"] + 1) if c["window"] else np.zeros_like(p)
        seen += int((p - low + 1).sum())
        touched += n - int(low[0])
    flops = 4 * seen * c["heads"] * dim
    io = 2 * sum(rows) * c["heads"] * dim * 2
    if c["op"] == "prompt":
        return {"bytes": io + touched * kv * dim * 4, "flops": flops}
    return {"bytes": io + touched * held + (touched * kv * 8 if c["weights"] else 0), "flops": flops}


# ------------------------------------------------- the definition in 64 bits
def _nibble64(x):
    """e2m1 from its bits: sign, two exponent bits with bias 1, one mantissa bit."""
    x = x.long()
    e, m = (x >> 1) & 3, x & 1
    mag = torch.where(e > 0, torch.ldexp((2 + m).double() / 2, (e - 1)), m.double() / 2)
    return torch.where(x >= 8, -mag, mag)


def _byte64(x):
    """E4M3 from its bits (no sign: scales)."""
    x = x.long()
    e, m = (x >> 3) & 15, x & 7
    return torch.where(e > 0, torch.ldexp((8 + m).double() / 8, e - 7), m.double() * 2.0 ** -9)


def _position64(s, table_row, head, positions):
    """K and V [n][dim] of some positions of one sequence and kv head, byte by byte from the layout's formula."""
    dim, ng = s["dim"], s["dim"] // 32
    tiles = s["page"] // 64
    p = positions.long()
    tile = (table_row.long()[p // s["page"]] * s["kv"] + head) * tiles + (p % s["page"]) // 64
    base, pos = (tile * ng * 2176)[:, None], (p % 64)[:, None]
    d = torch.arange(dim, device="cuda")[None, :]
    g = d // 32
    kc = s["cache"][base + g * 1024 + pos * 16 + (d % 32) // 2]
    ks = s["cache"][base + ng * 1024 + g * 64 + (pos % 16) * 4 + pos // 16]
    vc = s["cache"][base + ng * 1088 + (d // 16) * 512 + pos * 8 + (d % 16) // 2]
    vs = s["cache"][base + ng * 2112 + g * 64 + (pos // 4 % 4) * 16 + (pos // 16) * 4 + pos % 4]
    odd = (d % 2) * 4
    return _nibble64((kc.long() >> odd) & 15) * _byte64(ks), _nibble64((vc.long() >> odd) & 15) * _byte64(vs)


def _attend64(q, k, v, first, window, scale):
    """Row i of q (query position first + i // group rows at a time is the caller's) over k and v, all float64."""
    x = (q @ k.t()) * scale
    j = torch.arange(k.shape[0], device="cuda")[None, :]
    hide = j > first[:, None]
    if window:
        hide |= j <= first[:, None] - window
    x[hide] = -math.inf
    p = torch.softmax(x, 1)
    p = torch.where(hide.all(1, keepdim=True), torch.zeros_like(p), p)
    return p @ v, p


def _round64(x):
    x = x.double().reshape(*x.shape[:-1], -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    every = _byte64(torch.arange(0, 127, device="cuda"))
    scale = torch.zeros_like(top)
    for k in range(126, -1, -1):
        scale = torch.where(6.0 * every[k] >= top, every[k].expand_as(top), scale)
    scale = torch.where(top > 6.0 * 448.0, torch.full_like(top, 448.0), scale)
    r = torch.where(scale > 0, (x / torch.where(scale > 0, scale, torch.ones_like(scale))).abs(), torch.zeros_like(x))
    # e2m1: steps of a half below 2, of one below 4, of two above; round() takes ties to the even step
    mag = torch.where(r < 1.875, torch.round(2 * r) / 2, torch.where(r < 3.75, torch.round(r), 2 * torch.round(r / 2)))
    return (torch.sign(x) * mag.clamp(max=6.0) * scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    cached, rows = _lens(c)
    kv, dim = s["kv"], s["dim"]
    if c["op"] == "append":
        return _round64(s["k"]), _round64(s["v"])
    if c["op"] == "evict":
        ks, vs = [], []
        new = torch.zeros(s["weights_out"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(cached):
            kb, vb = [], []
            for h in range(kv):
                w = s["weights"][b, h, :n].cpu().numpy().astype(np.float64)
                if n > c["keep"]:
                    lo, hi = c["sinks"], n - c["recent"]
                    middle = np.lexsort((np.arange(lo, hi), -w[lo:hi]))[:c["keep"] - lo - c["recent"]] + lo
                    ids = np.sort(np.concatenate([np.arange(lo), middle, np.arange(hi, n)]))
                else:
                    ids = np.arange(n)
                new[b, h, :len(ids)] = torch.from_numpy(w[ids]).cuda()
                k, v = _position64(s, s["table"][b], h, torch.from_numpy(ids).cuda())
                kb.append(k)
                vb.append(v)
            ks.append(torch.stack(kb, 1))
            vs.append(torch.stack(vb, 1))
        return None, None, new, torch.cat(ks), torch.cat(vs)
    group = c["heads"] // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if c["op"] == "decode":
        total = s["weights"].double() if c["weights"] else None
        nq = c["q_rows"]
        for b, n in enumerate(cached):
            low = max(0, n - nq - c["window"] + 1) if c["window"] else 0   # nothing before it is seen
            if n == 0:
                continue
            first = torch.arange(n - nq, n, device="cuda").repeat_interleave(group) - low
            for h in range(kv):
                k, v = _position64(s, s["table"][b], h, torch.arange(low, n, device="cuda"))
                q = s["q"][b * nq:(b + 1) * nq, h * group:(h + 1) * group].double().reshape(nq * group, dim)
                o, p = _attend64(q, k, v, first, c["window"], s["scale"])
                out[b * nq:(b + 1) * nq, h * group:(h + 1) * group] = o.reshape(nq, group, dim)
                if total is not None:
                    total[b, h, low:n] += p.sum(0)
        return (out, total) if total is not None else out
    q0 = k0 = 0
    for p0, r in zip(cached, rows):
        n = p0 + r
        first = torch.arange(p0, n, device="cuda")
        for h in range(c["heads"]):
            k, v = (s[m][k0:k0 + n, h // group].double() for m in ("k", "v"))
            out[q0:q0 + r, h] = _attend64(s["q"][q0:q0 + r, h].double(), k, v, first, c["window"], s["scale"])[0]
        q0, k0 = q0 + r, k0 + n
    return out
