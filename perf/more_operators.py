"""Cases that time a serving step over the 4-bit key/value cache: its page tables and slot maps, attention of a chunk
of new tokens over the cached positions, and sparse attention over blocks that a cheap score selects.

Each case is one call (or the two calls that belong together) with data as a
serving program holds it: packed rows of q in 16 bits, a paged cache of e2m1
codes with one E4M3 scale per 32 values, page tables, lengths and row maps on
the GPU. Row i of sequence b is row cu_rows[b] + i of the packed rows and sits at
position start[b] + i. The plain form is elementary torch arithmetic in fp32 on
the same bytes; ``exact`` is the definition in float64, written apart from it.

Cache layout (one tile = 64 positions of one kv head; a page holds page / 64
tiles for each kv head, [kv_heads][page / 64][tile]); NG = head_dim / 32:
  K codes   16-byte chunk (pos, g)  at g * 1024 + pos * 16, low nibble = even k;
  K scales  byte (pos, g)           at NG * 1024 + g * 64 + (pos % 16) * 4 + pos / 16;
  V codes   8-byte chunk (pos, h)   at NG * 1088 + h * 512 + pos * 8, h = 16 values each;
  V scales  byte (pos, g)           at NG * 2112 + g * 64 + (pos / 4 % 4) * 16 + (pos / 16) * 4 + pos % 4.

Summaries of the cache's blocks (a block = one tile's 64 positions): [pages][kv_heads][page / 64] entries, first the
codes, head_dim int8 each, then for every entry one byte k. The mean key of a block is code * 2^(k - 16).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 sequences: a page now and then, a place for every token; given back after
        {"name": "plan_step", "op": "plan", "pieces": 0, "rows": 1, "singles": 64, "idle": 3, "page": 64, "len": 8000,
         "short": False},
        # a large step: many prompts enter beside running sequences, and the pool does not hold them all
        {"name": "plan_prompts", "op": "plan", "pieces": 150, "rows": 1900, "singles": 900, "idle": 40, "page": 64,
         "len": 4100, "short": True},
        # a short follow-up question behind a short context: only latency counts
        {"name": "chunk_short", "op": "chunk", "pieces": 1, "rows": 24, "singles": 0, "heads": 16, "kv_heads": 16,
         "dim": 64, "page": 64, "len": 201, "window": 0, "idle": 0, "type": "f16"},
        # a mixed step: a prompt's piece and the single tokens of sixteen running sequences, one slot idle
        {"name": "chunk_mixed", "op": "chunk", "pieces": 1, "rows": 512, "singles": 16, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 256, "len": 4000, "window": 0, "idle": 1, "type": "bf16"},
        # a few tokens behind a very long document, few kv heads
        {"name": "chunk_behind_long", "op": "chunk", "pieces": 1, "rows": 33, "singles": 0, "heads": 32, "kv_heads": 4,
         "dim": 128, "page": 256, "len": 65000, "window": 0, "idle": 0, "type": "f16"},
        # a long document's next piece
        {"name": "chunk_long", "op": "chunk", "pieces": 1, "rows": 2048, "singles": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 256, "len": 16384, "window": 0, "idle": 0, "type": "bf16"},
        # 32 sequences that each took sixteen tokens: the blocks that became full
        {"name": "blocks_step", "op": "blocks", "pieces": 32, "rows": 16, "singles": 0, "kv_heads": 8, "dim": 128,
         "page": 64, "len": 2000, "idle": 0},
        # six prompts that have just entered the cache
        {"name": "blocks_prompts", "op": "blocks", "pieces": 6, "rows": 8100, "singles": 0, "kv_heads": 8, "dim": 128,
         "page": 256, "len": 0, "idle": 0},
        # a decode step over long contexts chooses what each sequence will read
        {"name": "select_step", "op": "select", "pieces": 0, "rows": 1, "singles": 32, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 256, "len": 32768, "keep": 32, "sinks": 1, "recent": 2, "idle": 2, "type": "bf16"},
        # every token of a long document's piece chooses its own blocks
        {"name": "select_piece", "op": "select", "pieces": 1, "rows": 512, "singles": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 256, "len": 65000, "keep": 16, "sinks": 1, "recent": 2, "idle": 0, "type": "f16"},
        # the same step's attention over the chosen blocks
        {"name": "sparse_step", "op": "sparse", "pieces": 0, "rows": 1, "singles": 32, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 256, "len": 32768, "keep": 32, "idle": 2, "type": "bf16"},
        # and that of a piece, every token over its own blocks
        {"name": "sparse_piece", "op": "sparse", "pieces": 1, "rows": 512, "singles": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 256, "len": 65000, "keep": 16, "idle": 0, "type": "f16"},
    ]


def _log(rng, lo, hi):
    lo, hi = max(1, lo), max(lo, hi, 1)
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "chunk", "chunk", "chunk", "blocks", "select", "sparse", "sparse"])
    page = rng.choice([64, 128, 192, 256])
    if op == "plan":
        pieces, singles = _log(rng, 1, 200) - 1, _log(rng, 1, 2000)
        return {"op": op, "pieces": pieces, "rows": _log(rng, 2, 280000 // max(140, pieces)), "singles": singles,
                "idle": rng.choice([0, 1, singles // 20]), "page": page, "len": rng.randint(1, 8000),
                "short": rng.random() < 0.5}
    dim, kv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8, 8, 16])
    c = {"op": op, "kv_heads": kv, "dim": dim, "page": page, "singles": 0, "idle": 0}
    if op == "blocks":
        c["pieces"] = _log(rng, 1, 64)
        c.update(rows=_log(rng, 3, 32000 * 1024 // (c["pieces"] * kv * dim)), len=rng.randint(0, 2500))
        return c
    c.update(heads=kv * rng.choice([1, 2, 4, 5, 8]), type=rng.choice(["bf16", "f16"]))
    if op == "chunk":
        c["pieces"], c["singles"] = _log(rng, 1, 8), rng.choice([0, 0, 1, 3, 10])
        room = 1200000000 * 128 // (c["heads"] * (c["pieces"] + c["singles"]) * dim)   # rows times positions, padded
        c["rows"] = _log(rng, 2, min(2048, math.isqrt(room)))
        c["len"] = _log(rng, 30, min(65000, max(40, room // c["rows"] - c["rows"])))
        c.update(window=rng.choice([0, 0, 0, 900]), idle=rng.choice([0, 0, 1]))
        return c
    c["pieces"] = rng.choice([0, 0, 1, 2])
    c["singles"] = _log(rng, 1, 40) if c["pieces"] == 0 else rng.choice([0, 2])
    c["keep"] = _log(rng, 4, 64)
    batch = c["pieces"] + c["singles"]
    if op == "select":
        c["len"] = _log(rng, 300, min(131072, 12000000 * 128 * 8 // (batch * kv * dim)))
        c["rows"] = _log(rng, 2, min(512, 512 * 32 * 1024 * 64 // (c["len"] * c["heads"] * batch)))
        c.update(sinks=rng.choice([0, 1]), recent=rng.choice([1, 2, 3]))
    else:
        c["len"] = _log(rng, 300, min(131072, 1100000 * 128 * 8 // (batch * kv * dim)))
        room = 512 * 8 * 16 * 128 // (kv * dim)                                        # rows times blocks kept
        c["keep"] = max(2, min(c["keep"], room // max(1, c["singles"])))
        c["rows"] = _log(rng, 2, max(2, min(512, (room // c["keep"] - c["singles"]) // max(1, c["pieces"]))))
    return c


def _spread(batch, most, least=1):
    """Lengths of a ragged batch: the first is the longest, the others lie anywhere from an eighth of it up."""
    return [max(least, int(most * (1.0 - 0.875 * ((0.618034 * b) % 1.0)))) for b in range(batch)]


def _lens(case):
    """(positions before the step, new rows) of each sequence: pieces, then single tokens, some of those slots idle."""
    rows = _spread(case["pieces"], case["rows"]) + [1] * case["singles"]
    cached = _spread(len(rows), case["len"], 0)
    for i in range(case["idle"]):
        at = (len(rows) - 1 - 3 * i) % len(rows)
        rows[at] = 0
    return cached, rows


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


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)
    cached, rows = _lens(c)
    batch, page = len(rows), c["page"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c, "batch": batch, "page": page, "rows": sum(rows)}
    most = max(n + r for n, r in zip(cached, rows))
    columns = _ceil(max(most, 1), page)
    s["columns"], s["max_len"], s["max_rows"] = columns, most, max(rows)
    if c["op"] == "plan":
        held = [_ceil(n, page) for n in cached]
        new = [_ceil(n + r, page) - h for n, r, h in zip(cached, rows, held)]
        s["pages"] = sum(held) + sum(new) + 5
        order = torch.randperm(s["pages"], generator=g, device="cuda").to(torch.int32)
        there = torch.arange(columns, device="cuda") < ints(held)[:, None]
        s["table"] = torch.full((batch, columns), -1, dtype=torch.int32, device="cuda")
        s["table"][there] = order[:sum(held)]
        spare = (2 * sum(new)) // 3 if c["short"] else sum(new) + 5
        s["free"] = torch.full((s["pages"],), -1, dtype=torch.int32, device="cuda")
        s["free"][:spare] = order[sum(held):sum(held) + spare]
        s["count"] = ints([spare])
        s["lens"], s["want"] = ints(cached), ints(rows)
        new = lambda n, dt: torch.empty(n, dtype=dt, device="cuda")  # noqa: E731
        s["cu"], s["start"], s["lens_out"] = new(batch + 1, torch.int32), new(batch, torch.int32), new(batch, torch.int32)
        s["seq"], s["pos"], s["slot"] = new(s["rows"], torch.int32), new(s["rows"], torch.int32), new(s["rows"], torch.int64)
        return s
    kv, dim = c["kv_heads"], c["dim"]
    s["kv"], s["dim"], s["pages"] = kv, dim, batch * columns + 3
    s["cu"], s["start"] = ints(np.concatenate([[0], np.cumsum(rows)]).tolist()), ints(cached)
    s["table"], _ = _table(g, batch, columns, s["pages"])
    entries = s["pages"] * kv * (page // 64)
    if c["op"] == "select":
        # means of blocks: a part that blocks share and a part of their own, in the upper half of 7 bits
        mean = (22.0 * torch.randn(entries, dim, generator=g, device="cuda")).round().clamp(-127, 127)
        s["blocks"] = torch.cat([mean.to(torch.int8).view(-1).view(torch.uint8),
                                 torch.randint(9, 13, (entries,), generator=g, device="cuda", dtype=torch.uint8)])
        s["sel"] = torch.empty(s["rows"], kv, c["keep"], dtype=torch.int32, device="cuda")
    else:
        s["cache"] = _cache(g, s["pages"], kv, dim, page)
    if c["op"] == "blocks":
        s["blocks"] = torch.zeros(entries * (dim + 1), dtype=torch.uint8, device="cuda")
        return s
    s["scale"] = 1.0 / math.sqrt(dim)
    s["q"] = (2.0 * torch.randn(s["rows"], c["heads"], dim, generator=g, device="cuda")).to(TYPES[c["type"]])
    if c["op"] == "select":
        return s
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "sparse":
        at = np.concatenate([np.arange(n, n + r) for n, r in zip(cached, rows)])
        block = ints((at // 64).tolist())[:, None, None]
        n = columns * page // 64
        j = torch.arange(n, device="cuda")
        key = torch.rand(s["rows"], kv, n, generator=g, device="cuda")
        key = torch.where((j == 0) | ((j <= block) & (j >= block - 1)), key + 1.0, key).masked_fill(j > block, -1.0)
        best = key.topk(min(c["keep"], n), dim=-1)
        best = torch.where(best.values >= 0, best.indices, torch.full_like(best.indices, n)).sort(-1).values
        s["sel"] = torch.full((s["rows"], kv, c["keep"]), -1, dtype=torch.int32, device="cuda")
        s["sel"][..., :best.shape[-1]] = torch.where(best < n, best, torch.full_like(best, -1)).int()
    return s


# ------------------------------------------------------ the framework's calls
def _space(s, need):
    """A program asks once for its workspace, and keeps it."""
    if "ws" not in s:
        s["ws"] = torch.empty(need(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    from fp4_routed_expert_xp_amd import xp
    c = s["case"]
    if c["op"] == "plan":
        kd = xp.kv_dims(1, 64, s["page"], s["pages"])
        xp.xp_kv_plan(kd, s["lens"], s["want"], s["table"], s["free"], s["count"], s["cu"], s["start"], s["lens_out"],
                      s["seq"], s["pos"], s["slot"])
        xp.xp_kv_release(kd, s["lens_out"], s["lens"], s["table"], s["free"], s["count"])
        return s["cu"], s["start"], s["lens_out"], s["seq"], s["pos"], s["slot"], s["table"], s["free"], s["count"]
    kd = xp.kv_dims(s["kv"], s["dim"], s["page"], s["pages"])
    if c["op"] == "chunk":
        ws = _space(s, lambda: xp.xp_attn_chunk_workspace_bytes(kd, c["heads"], s["rows"], s["batch"], s["max_len"]))
        xp.xp_attn_chunk(kd, s["q"], s["cache"], s["table"], s["cu"], s["start"], s["max_len"], s["scale"], s["out"], ws,
                         window=c["window"])
        return s["out"]
    if c["op"] == "blocks":
        xp.xp_kv_blocks(kd, s["rows"], s["cu"], s["start"], s["table"], s["cache"], s["blocks"])
        if "parts" not in s:
            s["parts"] = _summaries(s)
        return s["parts"]
    if c["op"] == "select":
        xp.xp_attn_select(kd, s["q"], s["cu"], s["start"], s["table"], s["blocks"], s["sel"], sinks=c["sinks"],
                          recent=c["recent"])
        return s["sel"]
    ws = _space(s, lambda: xp.xp_attn_sparse_workspace_bytes(kd, c["heads"], s["rows"], c["keep"]))
    xp.xp_attn_sparse(kd, s["q"], s["cache"], s["table"], s["cu"], s["start"], s["sel"], s["scale"], s["out"], ws)
    return s["out"]


def _summaries(s):
    """The two parts of the summaries' buffer: codes (whole numbers) and the exponents beside them."""
    entries = s["pages"] * s["kv"] * (s["page"] // 64)
    codes = s["blocks"][:entries * s["dim"]].view(torch.int8).view(entries, s["dim"])
    return codes, s["blocks"][entries * s["dim"]:]


# ------------------------------------------------------------- plain forms
def _values(codes):
    """Code bytes [..., n] to the 2n values they stand for, without their scale."""
    lut = torch.tensor(E2M1, device=codes.device)
    return lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]


def _e4m3(b):
    return b.contiguous().view(torch.float8_e4m3fn).float()


def _keys(t, ng):
    """K [..., position][dim] of tiles t [..., bytes], fp32."""
    kc = _values(t[..., :ng * 1024].unflatten(-1, (ng, 64, 16)))
    ks = _e4m3(t[..., ng * 1024:ng * 1088]).unflatten(-1, (ng, 16, 4)).transpose(-1, -2).flatten(-2)
    return (kc * ks[..., None]).transpose(-3, -2).flatten(-2)


def _vals(t, ng):
    """V [..., position][dim] of tiles t [..., bytes], fp32."""
    vc = _values(t[..., ng * 1088:ng * 2112].unflatten(-1, (2 * ng, 64, 8)))
    vs = _e4m3(t[..., ng * 2112:]).unflatten(-1, (ng, 4, 4, 4)).transpose(-3, -2).flatten(-3)
    return (vc.unflatten(-3, (ng, 2)) * vs[..., None, :, None]).flatten(-4, -3).transpose(-3, -2).flatten(-2)


def _softmax(x, see):
    """Probabilities over the last axis among what `see` shows; rows that see nothing get zeros."""
    x = x.masked_fill_(~see, float("-inf"))
    e = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


def _place(s):
    """(sequence, row in it, position) of every packed row."""
    r = torch.arange(s["rows"], device="cuda")
    of = torch.searchsorted(s["cu"][1:], r, right=True)
    i = r - s["cu"][of]
    return of, i, s["start"][of] + i


def _plan(s):
    page, lens, want = s["page"], s["lens"].long(), s["want"].long()
    table, free, count = s["table"].flatten().clone(), s["free"].clone(), s["count"].long()
    need = (lens + want + page - 1) // page - (lens + page - 1) // page
    served = (want.cumsum(0) <= s["rows"]) & (need.cumsum(0) <= count)
    rows, need = want * served, need * served
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    cu, ends = torch.cat([zero, rows.cumsum(0)]), need.cumsum(0)
    # the j-th page taken: whose, which column of its table, and from where in the stack
    j = torch.arange(s["rows"] // page + s["batch"], device="cuda")
    of = torch.searchsorted(ends, j, right=True).clamp(max=s["batch"] - 1)
    at = of * s["columns"] + (lens[of] + page - 1) // page + j - (ends - need)[of]
    there = j < ends[-1]
    spill = torch.cat([table, zero.int()])               # one place more, for those that are not there
    spill[torch.where(there, at, torch.full_like(at, table.numel()))] = free[(count - 1 - j).clamp(min=0)]
    table = spill[:-1]
    r = torch.arange(s["rows"], device="cuda")
    of = torch.searchsorted(cu[1:], r, right=True).clamp(max=s["batch"] - 1)
    pos = lens[of] + r - cu[of]
    slot = table[of * s["columns"] + (pos // page).clamp(max=s["columns"] - 1)].long() * page + pos % page
    none = torch.full_like(r, -1)
    seq, pos, slot = (torch.where(r < cu[-1], v, none) for v in (of, pos, slot))
    # and back: from the last page to the first, on top of what is there
    count = count - ends[-1]
    column = torch.arange(s["columns"], device="cuda")
    go = (column >= ((lens + page - 1) // page)[:, None]) & (column < ((lens + rows + page - 1) // page)[:, None])
    go = go.flatten() & (table >= 0) & (table < s["pages"])
    rank = go.long().cumsum(0)
    spill = torch.cat([free, zero.int()])
    spill[torch.where(go, count + rank[-1] - rank, torch.full_like(rank, free.numel()))] = table
    table = torch.where(go, torch.full_like(table, -1), table)
    return (cu.int(), s["lens"], (lens + rows).int(), seq.int(), pos.int(), slot, table.view(s["batch"], -1), spill[:-1],
            (count + rank[-1]).int())


def _chunk(s):
    c, b, kv = s["case"], s["batch"], s["kv"]
    n64, ng = s["page"] // 64, s["dim"] // 32
    t = s["cache"].view(s["pages"], kv, n64, ng * 2176)[s["table"].int()].transpose(1, 2).flatten(2, 3)
    k, v = (f(t, ng).flatten(2, 3)[:, :, None] for f in (_keys, _vals))                  # [B][kv][1][position][dim]
    i, j = torch.arange(s["max_rows"], device="cuda"), torch.arange(k.shape[3], device="cuda")
    row = (s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"].float()[row].unflatten(2, (kv, -1)).permute(0, 2, 3, 1, 4)                # [B][kv][group][i][dim]
    x = torch.matmul(q * s["scale"], k.transpose(-1, -2).contiguous())
    at = (s["start"][:, None] + i)[:, :, None]
    see = j <= at
    see = see & (j > at - c["window"]) if c["window"] else see
    o = torch.matmul(_softmax(x, see[:, None, None]), v).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B][i][heads][dim]
    of, i, _ = _place(s)
    return o[of, i].to(s["q"].dtype)


def _tile_of(s, of, block):
    """Which tile of [pages][kv_heads][page / 64] block `block` of sequence `of` is, for kv head 0; kv heads follow n64 apart."""
    n64 = s["page"] // 64
    return s["table"][of, block // n64].long() * s["kv"] * n64 + block % n64


def _blocks(s):
    kv, ng, n64 = s["kv"], s["dim"] // 32, s["page"] // 64
    cached, rows = _lens(s["case"])                      # what a user's program knows: how many blocks there are at most
    most = max((n + r) // 64 - n // 64 for n, r in zip(cached, rows))
    first, end = s["start"] // 64, (s["start"] + s["cu"].diff()) // 64
    block = first[:, None] + torch.arange(most, device="cuda")
    there = block < end[:, None]
    of = torch.arange(s["batch"], device="cuda")[:, None]
    tile = _tile_of(s, of, block.clamp(max=s["columns"] * n64 - 1))[..., None] + n64 * torch.arange(kv, device="cuda")
    total = (_keys(s["cache"].view(-1, ng * 2176)[tile], ng).double() * 1024).sum(-2)   # whole numbers, [B][block][kv][dim]
    k = torch.arange(23, device="cuda")
    k = (total.abs().amax(-1, keepdim=True) > 127.0 * torch.exp2(k.double())).sum(-1)
    codes = torch.round(total * torch.exp2(-k.double())[..., None])
    entries = s["pages"] * kv * n64
    spill = [torch.cat([v, v[:1]]) for v in _summaries(s)]
    at = torch.where(there[..., None], tile, torch.full_like(tile, entries))
    spill[0][at] = codes.to(torch.int8)
    spill[1][at] = k.to(torch.uint8)
    return spill[0][:-1], spill[1][:-1]


def _select(s):
    c, kv, dim, keep = s["case"], s["kv"], s["dim"], s["case"]["keep"]
    n64, n = s["page"] // 64, s["columns"] * (s["page"] // 64)
    codes, k = _summaries(s)
    j = torch.arange(n, device="cuda")
    tile = _tile_of(s, torch.arange(s["batch"], device="cuda")[:, None], j)[:, None] + \
        n64 * torch.arange(kv, device="cuda")[:, None]                                    # [B][kv][block]
    q = s["q"].float()
    m, e = torch.frexp(q.abs().amax(-1, keepdim=True))
    e = e - 7 + (m > 127.0 / 128.0).int()
    q = torch.round(q * torch.exp2(-e.float()))                                           # [row][head][dim], whole numbers
    e = (e - e.unflatten(1, (kv, -1)).amax(2).repeat_interleave(c["heads"] // kv, 1)).float()
    i = torch.arange(s["max_rows"], device="cuda")
    row = (s["cu"][:-1, None] + i).clamp(max=s["rows"] - 1)
    pad = lambda v: v[row].unflatten(2, (kv, -1)).permute(0, 2, 3, 1, 4)  # noqa: E731    [B][kv][group][i][...]
    x = torch.matmul(pad(q), codes.float()[tile].transpose(-1, -2).contiguous()[:, :, None])
    x = x * torch.exp2(pad(e)) * torch.exp2(k.float())[tile][:, :, None, None]
    x = x.amax(2).transpose(1, 2)                                                         # [B][i][kv][block]
    of, i, at = _place(s)
    x, last = x[of, i], (at // 64)[:, None, None]
    x = torch.where((j < c["sinks"]) | (j > last - c["recent"]), torch.full_like(x, float("inf")), x)
    x = x.masked_fill(j > last, float("-inf"))
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(torch.arange(best.shape[-1], device="cuda") <= last, best, torch.full_like(best, n))
    best = torch.sort(best, dim=-1).values
    out = torch.full((s["rows"], kv, keep), -1, dtype=torch.int32, device="cuda")
    out[..., :best.shape[-1]] = torch.where(best < n, best, torch.full_like(best, -1)).int()
    return out


def _sparse(s):
    c, kv, ng, n64 = s["case"], s["kv"], s["dim"] // 32, s["page"] // 64
    of, _, at = _place(s)
    block = s["sel"].clamp(min=0).long()                                                  # [row][kv][keep]
    tile = _tile_of(s, of[:, None, None], block) + n64 * torch.arange(kv, device="cuda")[:, None]
    t = s["cache"].view(-1, ng * 2176)[tile]
    k, v = (f(t, ng).flatten(2, 3) for f in (_keys, _vals))                              # [row][kv][position][dim]
    p = (block[..., None] * 64 + torch.arange(64, device="cuda")).flatten(2)
    see = (p <= at[:, None, None]) & (s["sel"] >= 0).repeat_interleave(64, -1)
    q = s["q"].float().unflatten(1, (kv, -1)) * s["scale"]
    x = torch.matmul(q, k.transpose(-1, -2).contiguous())
    return torch.matmul(_softmax(x, see[:, :, None]), v).flatten(1, 2).to(s["q"].dtype)


def run(s):
    if own:
        return _own(s)
    return {"plan": _plan, "chunk": _chunk, "blocks": _blocks, "select": _select, "sparse": _sparse}[s["case"]["op"]](s)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    cached, rows = _lens(c)
    total = sum(rows)
    if c["op"] == "plan":
        new = sum(_ceil(n + r, c["page"]) - _ceil(n, c["page"]) for n, r in zip(cached, rows))
        # lengths in and out, a row's three places, pages from the stack to the tables and back
        return {"bytes": len(rows) * 20 + total * 16 + new * 16, "flops": 0}
    kv, dim = c["kv_heads"], c["dim"]
    half = kv * dim * 17 // 32          # bytes of one cached position's keys (or values): 4.25 bits each
    if c["op"] == "blocks":
        full = sum((n + r) // 64 - n // 64 for n, r in zip(cached, rows))
        return {"bytes": max(1, full) * (64 * half + kv * (dim + 1)), "flops": 0}
    width = total * c["heads"] * dim * 2
    if c["op"] == "select":
        seen = sum((n + r - 1) // 64 + 1 for n, r in zip(cached, rows) if r)
        dots = sum(int((np.arange(n, n + r) // 64 + 1).sum()) for n, r in zip(cached, rows))
        return {"bytes": width + seen * kv * (dim + 1) + total * kv * c["keep"] * 4, "flops": 2 * dots * c["heads"] * dim}
    if c["op"] == "sparse":
        tiles = pairs = 0
        for n, r in zip(cached, rows):
            if r:
                own_block = np.arange(n, n + r) // 64
                tiles += min(int(own_block[-1]) + 1, int(np.minimum(own_block + 1, c["keep"]).sum()))
                pairs += int((64 * np.minimum(own_block, c["keep"] - 1) + np.arange(n, n + r) % 64 + 1).sum())
        return {"bytes": 2 * width + total * kv * c["keep"] * 4 + tiles * 128 * half, "flops": 4 * pairs * c["heads"] * dim}
    seen = touched = 0
    for n, r in zip(cached, rows):
        if r:
            p = np.arange(n, n + r, dtype=np.int64)
            low = np.maximum(0, p - c["window"] + 1) if c["window"] else np.zeros_like(p)
            seen += int((p - low + 1).sum())
            touched += n + r - int(low[0])
    return {"bytes": 2 * width + touched * 2 * half, "flops": 4 * seen * c["heads"] * dim}


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


def exact(case, seed):
    if case["op"] in ("plan", "blocks", "select"):
        return None                                      # whole numbers
    s = prepare(case, seed)
    c = s["case"]
    cached, rows = _lens(c)
    group = c["heads"] // s["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    r0 = 0
    for b, (n, r) in enumerate(zip(cached, rows)):
        if c["op"] == "chunk" and r:
            low = max(0, n - c["window"] + 1) if c["window"] else 0       # nothing before it is seen
            at = torch.arange(n, n + r, device="cuda").repeat_interleave(group)[:, None] - low
            j = torch.arange(n + r - low, device="cuda")[None, :]
            hide = j > at
            if c["window"]:
                hide |= j <= at - c["window"]
            for h in range(s["kv"]):
                k, v = _position64(s, s["table"][b], h, torch.arange(low, n + r, device="cuda"))
                q = s["q"][r0:r0 + r, h * group:(h + 1) * group].double().reshape(r * group, -1)
                x = (q @ k.t()) * s["scale"]
                x[hide] = -math.inf
                out[r0:r0 + r, h * group:(h + 1) * group] = (torch.softmax(x, 1) @ v).view(r, group, -1)
        elif c["op"] == "sparse":
            lists = s["sel"][r0:r0 + r].cpu().numpy()
            for i in range(r):
                for h in range(s["kv"]):
                    p = (lists[i, h][lists[i, h] >= 0][:, None] * 64 + np.arange(64)).reshape(-1)
                    p = torch.from_numpy(p[p <= n + i]).cuda()
                    k, v = _position64(s, s["table"][b], h, p)
                    q = s["q"][r0 + i, h * group:(h + 1) * group].double()
                    out[r0 + i, h * group:(h + 1) * group] = torch.softmax((q @ k.t()) * s["scale"], 1) @ v
        r0 += r
    return out
