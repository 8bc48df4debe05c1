"""Attention of equal scores over values that name their tile: which positions took part, and how often.

All keys are alike, so a row's weights are 1 / n each. v is 0 but for one column of each tile of 64
positions: tile t holds VALUES[t / dim mod 6] in column t mod dim. Exponentials and sums are whole
multiples of powers of two below 2^24 times them, hence exact in fp32, and a row's output is the
tiles' counts times their values over n, rounded twice in fp32 and once to fp16."""
import numpy as np

CODES = np.array([2, 4, 6, 7, 5, 3], dtype=np.uint8)                 # e2m1 of
VALUES = np.array([1.0, 2.0, 4.0, 6.0, 3.0, 1.5])
REL = 2.0 ** -11 + 2.0 ** -22                                        # half a step of fp16, two roundings of fp32


def column(tile, dim):
    return tile % dim, (tile // dim) % len(VALUES)


def counts(at, window):
    """How many positions of each tile a row at position `at` sees."""
    if at < 0:
        return np.zeros(0)
    lo = max(0, at - window + 1) if window else 0
    t = np.arange(at // 64 + 1)
    return np.maximum(0, np.minimum(64 * t + 64, at + 1) - np.maximum(64 * t, lo)).astype(np.float64)


def output(c, dim):
    """The output of a row that sees c[t] positions of tile t."""
    out = np.zeros(dim)
    col, val = column(np.arange(len(c)), dim)
    np.add.at(out, col, c * VALUES[val])
    return out / max(c.sum(), 1.0)


def not_told_apart(c, dim):
    """The tiles a row sees that may be left out or doubled without moving its output beyond REL."""
    want, tiles = output(c, dim), []
    for t in np.nonzero(c)[0]:
        for times in (0.0, 2.0):
            d = c.copy()
            d[t] *= times
            if (np.abs(output(d, dim) - want) <= REL * want).all():
                tiles.append(int(t))
    return tiles


def _ragged(batch, short, **longer):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, short, batch)
    for b, n in longer.items():
        lens[int(b[1:])] = n
    return lens.tolist()


# kv heads, heads of each, dim, page, tokens a sequence, window, lengths, max_len
DECODE = {
    "one_of_17000_among_512_units": (8, 1, 64, 64, 1, 0, _ragged(64, 130, s17=17000), 17000),
    "one_of_16000_whole_among_512_units": (8, 1, 64, 64, 1, 0, _ragged(64, 130, s17=16000), 16000),
    "two_long_of_64": (1, 3, 64, 64, 2, 0, _ragged(64, 130, s32=11000, s63=3300), 12000),
    "two_long_of_70": (1, 3, 64, 64, 2, 0, _ragged(70, 130, s35=11000, s69=3300), 12000),
    "two_long_of_130_sized_for_100": (1, 3, 64, 64, 2, 0, _ragged(130, 130, s65=11000, s129=3300), 100),
    "two_long_of_9": (1, 3, 64, 64, 2, 0, _ragged(9, 130, s4=11000, s8=3300), 12000),
    "300_sequences_in_order_of_length": (1, 4, 128, 128, 1, 0, _ragged(300, 700, s5=4000), 300),
    "64_sequences_in_classes_of_length": (5, 2, 64, 64, 1, 0, _ragged(64, 2000), 1000),
    "one_long": (4, 8, 128, 256, 1, 0, [131072], 131072),
    "one_long_of_256_columns": (2, 8, 256, 64, 1, 0, [40000], 40000),
    "forty_rows_a_head": (2, 8, 128, 128, 5, 0, [9000, 777], 9000),
    "forty_rows_a_head_of_256_columns": (2, 8, 256, 128, 5, 0, [5000, 777], 5000),
    "window": (2, 8, 128, 192, 5, 2100, [9000, 2099, 777], 9000),
    "window_of_cut_sequences": (1, 4, 64, 64, 3, 7000, [20000, 6000], 20000),
    "whole": (3, 4, 128, 64, 1, 0, [1, 63, 64, 65, 900], 900),
}

# kv heads, heads of each, dim, queries, keys, window
PROMPT = {
    "few_64": (1, 2, 64, [200, 70], [5000, 300], 0), "few_128": (1, 2, 128, [200, 70], [5000, 300], 0),
    "256": (1, 1, 256, [200, 70], [5000, 300], 0), "many_64": (64, 2, 64, [200, 130], [3000, 300], 0),
    "many_128": (64, 2, 128, [200, 130], [3000, 300], 0), "whole_prompt": (1, 1, 64, [2500], [2500], 0),
    "window": (1, 3, 128, [200, 70], [5000, 300], 1500),
}


def decode_rows(case):
    """(sequence, token, position) of a case's rows."""
    _, _, _, _, q_rows, _, lens, _ = case
    return [(b, i, n - q_rows + i) for b, n in enumerate(lens) for i in range(q_rows)]


def prompt_rows(case):
    """(row, position) of a case's query tokens."""
    _, _, _, nq, nk, _ = case
    return list(enumerate(m - n + i for n, m in zip(nq, nk) for i in range(n)))
