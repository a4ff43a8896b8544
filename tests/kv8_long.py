"""Inputs of the long-context KV8 tests, and what they are compared with."""
import numpy as np

from oracle import serving_oracle as S

UNIT = 32  # tokens of a decode tile, a quarter of a prefill tile


def paged(lens, P, rng):
    """A block table with every sequence's pages in any order of a pool without spare pages."""
    need = [-(-int(n) // P) for n in lens]
    order = rng.permutation(sum(need))
    table = np.full((len(lens), max(need)), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
    return table, sum(need)


def case(Hq, Hkv, P, new, old, seed, keys, values):
    """(q, codes, scales, table, lens, start); keys and values: (rng, L, Hkv) -> int8
    codes [L, Hkv, 128] of a sequence."""
    rng = np.random.default_rng(seed)
    lens = np.asarray([n + o for n, o in zip(new, old)], np.int32)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, pages = paged(lens, P, rng)
    codes = rng.integers(-127, 128, (pages, 2, Hkv, P, 128)).astype(np.int8)  # also behind the sequences' ends
    for b, L in enumerate(lens):
        for kv, make in enumerate((keys, values)):
            x = np.zeros((-(-L // P) * P, Hkv, 128), np.int8)
            x[:L] = make(rng, int(L), Hkv)
            x[L:] = 99
            codes[table[b, :-(-L // P)], kv] = x.reshape(-1, P, Hkv, 128).transpose(0, 2, 1, 3)
    scales = np.full((pages, 2, Hkv), 0.02, np.float32)
    q = (rng.standard_normal((int(start[-1]), Hq, 128)) * 0.5).astype(np.float16)
    return q, codes, scales, table, lens, start


def random_codes(rng, L, Hkv):
    return np.clip(np.rint(rng.standard_normal((L, Hkv, 128)) * 35), -127, 127).astype(np.int8)


def marked(rng, L, Hkv):
    """Values that are 0 but for one dimension of one kv head in each unit of 32
    tokens: what a dimension of the output is, its units alone have made."""
    u = np.arange(L) // UNIT % (128 * Hkv)
    x = np.zeros((L, Hkv, 128), np.int8)
    x[np.arange(L), u // 128, u % 128] = 127
    return x


def check_rows(c, y, scale, weight_eps, weight_floor, rows=None, heads=None):
    """Rows (all of the batch if None) of y against the oracle's bound and half an fp16
    ulp; returns the largest |error| / bound."""
    q, codes, scales, table, lens, start = c
    worst = 0.0
    hs = list(range(q.shape[1]) if heads is None else heads)
    for r in range(int(start[-1])) if rows is None else rows:
        b = int(np.searchsorted(start, r, side="right")) - 1
        limit = int(lens[b]) - int(start[b + 1]) + r + 1
        o, E = S.attention(q[r:r + 1], codes, scales, table[b:b + 1], [limit], [0, 1], scale, weight_eps, hs, weight_floor)
        o, E, got = o[0, hs], E[0, hs], y[r, hs].astype(np.float64)
        ulp = np.spacing(np.maximum(np.abs(o) + E, 6.2e-5).astype(np.float16)).astype(np.float64)
        assert np.isfinite(got).all()
        bad = np.abs(got - o) / (0.5 * ulp + E)
        worst = max(worst, float(bad.max()))
    return worst
