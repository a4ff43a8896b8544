"""The paged 8-bit KV cache at the ends of its documented ranges: the most
sequences, the longest sequence, the largest query groups, caches whose offsets
pass 32 bits.

Tolerances: half an fp16 ulp and an evaluation bound. Where a sequence is too
long for the oracle's (2 L roundings), the kernels' own depth is counted: see
`longest`.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from oracle import serving_oracle as S  # noqa: E402
from tests import kv8_long as K  # noqa: E402
from tests.test_gpu_kv8 import DEV, SCALE, _no_device_error, attend, case, check_attention, dev, host  # noqa: E402,F401


def half_ulp(y):
    return 0.5 * np.spacing(np.maximum(np.abs(y), 6.2e-5).astype(np.float16)).astype(np.float64)


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (1024, 1), (1024, 1024), (512, 8)])
def test_largest_groups_and_head_counts(Hq, Hkv):
    c = case(Hq, Hkv, 16, [1, 1], [299, 40], 3)
    check_attention(c, attend(c, True), 2.0 ** -20, heads=(0, 1, Hq // 2, Hq - 1))
    c = case(Hq, Hkv, 16, [1, 3, 0, 2], [70, 300, 5, 0], 4, pad_rows=1)
    check_attention(c, attend(c, False), 2.0 ** -11, heads=(0, 1, Hq // 2, Hq - 1))


def test_the_most_sequences():
    """65535 sequences of 0 to 2 tokens, each in a page of its own: attention over one token is its value."""
    B, P = 65535, 16
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 3, B).astype(np.int32)
    qkv = rng.standard_normal((B, 3, 128)).astype(np.float16)
    codes, scales = w4a8.kv8_cache(B, 1, P, DEV)
    table = dev(rng.permutation(B).astype(np.int32)[:, None])
    f, _ = w4a8.rope_frequencies(128, device=DEV)
    q = torch.full((B, 1, 128), 7.0, dtype=torch.float16, device=DEV)
    for step in (1, 2):  # the first tokens, then the second ones
        now = dev(np.where(lens >= step, step, 0).astype(np.int32))
        w4a8.kv8_rope_append(dev(qkv.reshape(B, -1)), 1, codes, scales, table, now, f, out=q)
    y = host(w4a8.kv8_attention_decode(q, codes, scales, table, dev(lens), SCALE))
    start = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    some = torch.from_numpy(lens).to(DEV).clamp(min=1)  # (a row of a sequence needs a token)
    y2 = host(w4a8.kv8_attention_prefill(q, codes, scales, table, some, start, SCALE))
    assert not y[lens == 0].any() and (host(q)[lens == 0] == 7).all()
    hc, hs, ht = host(codes), host(scales), host(table)[:, 0]
    V = hc[ht, 1, 0, :2].astype(np.float64) * hs[ht, 1, 0].astype(np.float64)[:, None, None]
    for got, which in ((y, lens == 1), (y2, lens <= 1)):
        want = V[which, 0]
        assert (np.abs(got[which, 0] - want) <= half_ulp(want) + 2.0 ** -19 * np.abs(want)).all()
    for b in np.flatnonzero(lens == 2)[:200]:
        o, E = S.attention(host(q[b:b + 1]), hc, hs, ht[b:b + 1, None], [2], [0, 1], SCALE, 2.0 ** -11)
        for got in (y, y2):
            assert (np.abs(got[b] - o[0]) <= half_ulp(np.abs(o[0]) + E[0]) + E[0]).all()


@pytest.mark.parametrize("P", [16, 128])
def test_offsets_that_pass_32_bits(P):
    """A cache of more than 6 GB, its first and last pages in use."""
    Hkv = 8
    pages = (6 << 30) // (2 * Hkv * P * 128)
    codes, scales = w4a8.kv8_cache(pages, Hkv, P, DEV)
    rng = np.random.default_rng(8)
    old, new = [5, 3 * P - 1], [2 * P, P + 3]
    lens = np.asarray(old, np.int32) + np.asarray(new, np.int32)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    wide = -(-int(lens.max()) // P)
    used = np.concatenate([np.arange(wide), pages - 1 - np.arange(wide)])
    table = rng.permutation(used).reshape(2, wide).astype(np.int32)
    f, _ = w4a8.rope_frequencies(128, device=DEV)
    T = int(start[-1])
    # the tokens cached before, then the new ones, in two calls
    q = None
    for a, n in ((np.zeros(2, int), old), (np.asarray(old), new)):
        at = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        qkv = rng.standard_normal((int(at[-1]), 3 * Hkv, 128)).astype(np.float16)
        q = w4a8.kv8_rope_append(dev(qkv.reshape(len(qkv), -1)), Hkv, codes, scales, dev(table), dev((a + n).astype(np.int32)), f,
                                 q_start=dev(at))
    # the pages in use, as a small cache of their own
    small = np.unique(table)
    hc, hs = host(codes[torch.from_numpy(small).to(DEV).long()]), host(scales[torch.from_numpy(small).to(DEV).long()])
    ht = np.searchsorted(small, table).astype(np.int32)
    assert hc.any(axis=(1, 2, 3, 4))[ht[:, 0]].all()
    untouched = torch.ones(pages, dtype=torch.bool, device=DEV)
    untouched[torch.from_numpy(small).to(DEV).long()] = False
    assert not scales[untouched].any()
    y = w4a8.kv8_attention_prefill(q, codes, scales, dev(table), dev(lens), dev(start), SCALE)
    c = (host(q), hc, hs, ht, lens, start)
    rows = sorted({0, T - 1, new[0] - 1, new[0], *rng.integers(0, T, 8).tolist()})
    assert K.check_rows(c, host(y), SCALE, 2.0 ** -11, 2.0 ** -35, rows=rows, heads=(0, 3, 7)) <= 1
    last = [new[0] - 1, T - 1]
    yd = w4a8.kv8_attention_decode(q[last].contiguous(), codes, scales, dev(table), dev(lens), SCALE)
    cd = (host(q)[last], hc, hs, ht, lens, np.asarray([0, 1, 2], np.int32))
    assert K.check_rows(cd, host(yd), SCALE, 2.0 ** -20, 2.0 ** -39) <= 1


def longest(q, codes, scales, table, L, h, G):
    """(y, a) of one row over L tokens of pages named many times: each distinct page counted as often as it stands."""
    P = codes.shape[3]
    times = np.bincount(table[0, :L // P], minlength=len(codes)).astype(np.float64)
    k = codes[:, 0, h // G].astype(np.float64) * scales[:, 0, h // G].astype(np.float64)[:, None, None]
    v = codes[:, 1, h // G].astype(np.float64) * scales[:, 1, h // G].astype(np.float64)[:, None, None]
    s = SCALE * (k.reshape(-1, 128) @ q.astype(np.float64))
    p = np.exp(s - s.max()) * np.repeat(times, P)
    p /= p.sum()
    return p @ v.reshape(-1, 128), p @ np.abs(v.reshape(-1, 128))


@pytest.mark.parametrize("n,Hq", [(0, 2), (1, 5), (40, 1)])
def test_the_longest_sequence(n, Hq):
    """2^24 tokens in 131072 places of a table that names seven pages. n = 0: the decode call.

    Depth of the kernels' sums. Decode: 524288 tiles over at least 148 x 8 warps are under 450 tiles a warp, each with 2
    accumulations of the output and 4 of the denominator, then 24 partial results of a CTA and 148 CTAs: under 3000
    roundings in all. Prefill: 131072 tiles of 128 tokens in 32 parts, 4096 tiles a part with 8 accumulations and 4: under
    2^15 + 2^14 + 300. Each is off by 2^-23 of sum p |V| at most. The weights by 2^-20, 2^-11 (prefill); the scores by the
    oracle's delta, 131 * 2^-23 * scale * sK * sum |q c| <= 40 * 2^-16, in numerator and denominator."""
    P, L = 128, 1 << 24
    rng = np.random.default_rng(9)
    codes = np.clip(np.rint(rng.standard_normal((7, 2, 1, P, 128)) * 35), -127, 127).astype(np.int8)
    codes[:, 1] |= 1  # (no sum of values cancels to nothing)
    codes[:, 1] = np.abs(codes[:, 1].astype(np.int16)).clip(1, 127).astype(np.int8)
    scales = np.full((7, 2, 1), 0.02, np.float32)
    table = rng.integers(0, 7, (1, L // P)).astype(np.int32)
    rows = max(n, 1)
    q = (rng.standard_normal((rows, Hq, 128)) * 0.5).astype(np.float16)
    g = [dev(a) for a in (q, codes, scales, table, np.asarray([L], np.int32))]
    if n == 0:
        y = w4a8.kv8_attention_decode(*g, SCALE)
    else:
        y = w4a8.kv8_attention_prefill(*g, torch.tensor([0, n], dtype=torch.int32, device=DEV), SCALE)
    y = host(y).astype(np.float64)
    few = n * Hq <= 32
    rel = (3000 if few else 2 ** 15 + 2 ** 14 + 300) * 2.0 ** -23 + (2.0 ** -20 if few else 2.0 ** -11) + 80 * 2.0 ** -16
    scores = SCALE * 0.02 * np.einsum("td,rhd->rht", codes[:, 0, 0].reshape(-1, 128).astype(np.float64), q.astype(np.float64))
    assert SCALE * 0.02 * (np.abs(codes[:, 0, 0].reshape(-1, 128).astype(np.float64)) @ np.abs(q[0, 0].astype(np.float64))).max() < 40
    for i in {0, rows - 1}:
        for h in range(Hq):
            want, a = longest(q[i, h], codes, scales, table, L, h, Hq)
            # an earlier row does not see the last tokens: their share of the sum at most, in numerator and denominator
            share = (rows - 1 - i) * np.exp(scores[i, h].max() - scores[i, h].min()) / L
            assert (np.abs(y[i, h] - want) <= half_ulp(want) + (rel + 2 * share) * a).all()
