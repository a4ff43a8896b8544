"""KV8 attention over long contexts, where no tile may be lost: every dimension
of the output made by a few units of 32 tokens alone (the bound rejects an
output without one of them: tests/test_serving_bounds.py), scores that grow or
fall along the cache, both instantiations of the prefill kernel with both
blocks of rows at work.

Tolerances: the oracle's bound and half an fp16 ulp, as in tests/test_gpu_kv8.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests import kv8_long as K  # noqa: E402
from tests.test_gpu_kv8 import DEV, SCALE, _no_device_error, attend, dev  # noqa: E402,F401

DECODE, PREFILL = (2.0 ** -20, 2.0 ** -39), (2.0 ** -11, 2.0 ** -35)


def cut(c):
    """Whether the batch's pieces of 256 rows are cut along the cache: while they fill half of 148 SMs at most."""
    q, codes, _, _, lens, _ = c
    Hkv = codes.shape[2]
    return (q.shape[0] * (q.shape[1] // Hkv) // 256 + len(lens)) * Hkv * 2 <= 148


def growing(sign):
    """Keys along the queries' common direction, whose scores grow (or fall) by
    about 68 in powers of e over the cache: SCALE * 0.02 * 128 * 2.5 * 120."""
    def make(rng, L, Hkv):
        step = np.arange(L) / max(L - 1, 1) if sign > 0 else 1 - np.arange(L) / max(L - 1, 1)
        return np.clip(np.rint(step[:, None, None] * 120 + rng.standard_normal((L, Hkv, 128)) * 3), -127, 127).astype(np.int8)
    return make


def aligned_queries(c):
    """Queries of about 2.5 in every dimension: scores along the keys' common direction."""
    q = np.random.default_rng(3).standard_normal(c[0].shape) * 0.05 + 2.5
    return (q.astype(np.float16),) + tuple(c[1:])


# ------------------------------------------------------------------- decode
@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 1, [20000, 1, 70, 3999]), (4, 1, [20000]), (16, 8, [8192, 8191, 33, 12001]),
                                         (64, 8, [5000, 9017]), (64, 64, [4096, 2100]), (12, 1, [9000])])
@pytest.mark.parametrize("P", [16, 64])
def test_decode_loses_no_unit(Hq, Hkv, lens, P):
    c = K.case(Hq, Hkv, P, [1] * len(lens), [n - 1 for n in lens], Hq + P, K.random_codes, K.marked)
    heads = range(0, Hq, max(Hq // Hkv, 1)) if Hq > 8 else range(Hq)
    assert K.check_rows(c, attend(c, True), SCALE, *DECODE, heads=heads) <= 1


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 1), (32, 8)])
def test_decode_of_growing_and_falling_scores(sign, Hq, Hkv):
    c = aligned_queries(K.case(Hq, Hkv, 32, [1, 1], [8999, 700], 5, growing(sign), K.random_codes))
    assert K.check_rows(c, attend(c, True), SCALE, *DECODE, heads=(0, Hq - 1)) <= 1


# ------------------------------------------------------------------ prefill
def sampled(c, n=7):
    """First and last rows of each sequence, rows at the edges of the blocks of 128 and pieces of 256, and some others."""
    q, codes, _, _, _, start = c
    G = q.shape[1] // codes.shape[2]
    rows = set()
    for b in range(len(start) - 1):
        a, e = int(start[b]), int(start[b + 1])
        if a == e:
            continue
        rows |= {a, e - 1, min(a + 127 // G, e - 1), min(a + 128 // G, e - 1), min(a + 256 // G, e - 1)}
        rows |= set(np.random.default_rng(e).integers(a, e, n).tolist())
    return sorted(rows)


LONG = [((32, 8, 16, [1000], [8017]), False),            # a chunk over a long context: whole pieces, 64 to 71 tiles
        ((32, 8, 64, [1500, 2100, 1800], [0, 0, 0]), False),  # new prompts: whole pieces, 1 to 17 tiles
        ((48, 3, 32, [333, 420], [3000, 900]), False),   # 16 heads a kv head: 21 and 27 pieces of a head
        ((32, 8, 64, [200, 20], [20000, 300]), True),    # pieces cut along the cache
        ((4, 1, 16, [700], [9000]), True),
        ((3, 1, 128, [300, 2], [12345, 60]), True)]


@pytest.mark.parametrize("shape,is_cut", LONG)
def test_prefill_loses_no_unit(shape, is_cut):
    Hq, Hkv = shape[:2]
    c = K.case(*shape, 40 + Hq, K.random_codes, K.marked)
    assert cut(c) == is_cut
    y = attend(c, False)
    heads = sorted({0, Hq // Hkv - 1, Hq // 2, Hq - 1})
    assert K.check_rows(c, y, SCALE, *PREFILL, rows=sampled(c), heads=heads) <= 1


@pytest.mark.parametrize("shape,is_cut", LONG)
def test_prefill_of_long_contexts(shape, is_cut):
    """Ordinary values; the same bits every time."""
    Hq, Hkv = shape[:2]
    c = K.case(*shape, 50 + Hq, K.random_codes, K.random_codes)
    assert cut(c) == is_cut
    y = attend(c, False)
    assert K.check_rows(c, y, SCALE, *PREFILL, rows=sampled(c, 3), heads=(0, Hq - 1)) <= 1
    g = [dev(a) for a in c]
    ref, out = dev(y).view(torch.int16), torch.empty_like(g[0])
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(30):
        w4a8.kv8_attention_prefill(*g, SCALE, out=out)
        bad += (out.view(torch.int16) != ref).any()
    assert int(bad) == 0


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shape,is_cut", [LONG[0], LONG[1], LONG[4]])
def test_prefill_of_growing_and_falling_scores(shape, is_cut, sign):
    """The reference moves in every few tiles, or never after the first."""
    Hq = shape[0]
    c = aligned_queries(K.case(*shape, 60 + Hq, growing(sign), K.random_codes))
    assert cut(c) == is_cut
    assert K.check_rows(c, attend(c, False), SCALE, *PREFILL, rows=sampled(c, 3), heads=(0, Hq - 1)) <= 1
