"""GPU: every position that a row sees takes part in its attention once, however a batch is cut into pieces,
ordered and joined (attn_tiles.py; the host tests show that its bound tells any one tile left out or doubled)."""
import numpy as np
import pytest
import torch

from fp4_routed_expert_xp_amd import xp

import attn_ref as ref
import attn_tiles as at
from test_gpu_attn import dev, dims_of, ends, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("name", at.DECODE)
def test_decode_sees_every_position_once(name, weights):
    case = at.DECODE[name]
    kv, group, dim, page, q_rows, window, lens, max_len = case
    cols = -(-max(lens) // page)
    used = [-(-n // page) for n in lens]
    rng = np.random.default_rng(1)
    ids = rng.permutation(sum(used) + 3)
    c = ref.Cache(kv, dim, page, len(ids), rng=rng)        # what no sequence holds is anything
    table, first = np.full((len(lens), cols), -1, dtype=np.int32), 0
    for b, u in enumerate(used):
        table[b, :u] = ids[first:first + u]
        first += u
    ng, pos = dim // 32, np.arange(64)
    for b, u in enumerate(used):
        for p in range(u):
            for i in range(page // 64):
                t = c.b[table[b, p], :, i]
                t[:, :ng * 1024] = 0x22                    # every key is 1 in every column
                t[:, ng * 1088:ng * 2112] = 0
                t[:, ng * 1024:ng * 1088] = t[:, ng * 2112:] = 0x38
                col, val = at.column(p * (page // 64) + i, dim)
                t[:, ng * 1088 + (col // 16) * 512 + pos * 8 + (col % 16) // 2] = at.CODES[val] << (4 * (col % 2))
    for b, n in enumerate(lens):                           # what lies behind a sequence's end is NaN
        if n % page:
            for i in range(page // 64):
                behind = pos[i * 64 + pos >= n % page]
                for g in range(ng):
                    at_v = ng * 2112 + g * 64 + (behind // 4 % 4) * 16 + (behind // 16) * 4 + behind % 4
                    c.b[table[b, n // page], :, i, at_v] = 0x7f
                    c.b[table[b, n // page], :, i, ng * 1024 + g * 64 + (behind % 16) * 4 + behind // 16] = 0x7f
    d = dims_of(c)
    q = dev(rng.normal(size=(len(lens) * q_rows, kv * group, dim)), torch.float16)
    out = torch.full_like(q, 3.0)
    w = torch.zeros(len(lens), kv, cols * page, device="cuda") if weights else None
    ws = torch.empty(xp.xp_attn_decode_workspace_bytes(d, kv * group, q_rows, len(lens), max_len), dtype=torch.uint8,
                     device="cuda")
    xp.xp_attn_decode(d, q, torch.from_numpy(c.b.reshape(-1)).cuda(), dev(table), ints(lens), max_len, 0.125, out, ws,
                      q_rows=q_rows, window=window, weights=w)
    got = out.double().cpu().numpy()
    sums = np.zeros((len(lens), cols * page))
    for b, i, place in at.decode_rows(case):
        want = at.output(at.counts(place, window), dim)
        err = np.abs(got[b * q_rows + i] - want)
        assert (err <= at.REL * want).all(), (b, i, place, float(err.max()))
        lo = max(0, place - window + 1) if window else 0
        if place >= 0:
            sums[b, lo:place + 1] += group / (place + 1 - lo)
    if weights:                                            # each a product of two rounded numbers, added up
        w = w.double().cpu().numpy()
        assert (np.abs(w - sums[:, None]) <= (q_rows * group + 3) * 2.0 ** -24 * sums[:, None]).all()


@pytest.mark.parametrize("name", at.PROMPT)
def test_prompt_sees_every_position_once(name):
    case = at.PROMPT[name]
    kv, group, dim, nq, nk, window = case
    cu_q, cu_k = ends(nq), ends(nk)
    rng = np.random.default_rng(2)
    v = np.zeros((cu_k[-1], kv, dim))
    for b, n in enumerate(nk):
        col, val = at.column(np.arange(n) // 64, dim)
        v[cu_k[b] + np.arange(n), :, col] = at.VALUES[val][:, None]
    q = dev(rng.normal(size=(cu_q[-1], kv * group, dim)), torch.float16)
    k, v = torch.ones(v.shape, dtype=torch.float16, device="cuda"), dev(v, torch.float16)
    out = torch.full_like(q, 3.0)
    xp.xp_attn_prompt(q, k, v, dev(cu_q), dev(cu_k), 0.125, out, window=window)
    got = out.double().cpu().numpy()
    for row, place in at.prompt_rows(case):
        want = at.output(at.counts(place, window), dim)
        err = np.abs(got[row] - want)
        assert (err <= at.REL * want).all(), (row, place, float(err.max()))
