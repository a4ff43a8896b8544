"""The paged 8-bit KV cache: rotation and append, decode and prefill
attention, against the oracle in 64 bits.

Tolerances, derived. Append: the sine and cosine are within 2^-20.5 (their
angle within 2^-22), so a rotated value is within 2^-19.5 of its pair's larger
half, under 2 ROT, scale factor included; a page's scale is within 2 ROT of the
exact one relatively; with the scale taken as given a new code is within 1/2
+ 127 * 4 ROT of x / s', a carried code within 1/2 + 127 * 2^-22. Attention:
the oracle's bound plus half an fp16 ulp; the decode kernels keep the
softmax weights to 2^-20, the prefill kernel rounds them to fp16 (2^-11).
Both hold them in fp16 with the largest at 2^14 (decode, two terms) or at
least 2^10 (prefill), where the smallest step is 2^-24: a rounding there is
off by 2^-25, i.e. by 2^-39 or 2^-35 of the largest weight, however small the
weight itself (the floor of the bound).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8
from w4a8_quantized_gemm_quantize_b200 import inputs as I
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
SCALE = float(np.float32(1.0 / np.sqrt(128.0)))
ROT = 2.0 ** -20


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.cpu().numpy()


def i32(a):
    return np.asarray(a, np.int32)


@pytest.fixture(autouse=True)
def _no_device_error():
    w4a8.clear_device_error(DEV)
    yield
    assert w4a8.get_device_error(DEV) == 0


def paged(lens, P, rng, spare=3, wide=0, first=None):
    """A block table with the pages of each sequence (from position first[b]
    on) in any order of a pool; the other entries are not looked at."""
    lo = [0] * len(lens) if first is None else [int(n) // P for n in first]
    need = [max(-(-int(n) // P) - a, 0) for n, a in zip(lens, lo)]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(-(-int(n) // P) for n in lens), 1) + wide), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, lo[b]:lo[b] + n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def random_cache(pages, Hkv, P, rng):
    """Codes and scales as quantized pages have them: each page and head with its own range."""
    codes = np.clip(np.rint(rng.standard_normal((pages, 2, Hkv, P, 128)) * 35), -127, 127).astype(np.int8)
    scales = np.exp(rng.uniform(np.log(0.005), np.log(0.1), (pages, 2, Hkv))).astype(np.float32)
    return codes, scales


# ------------------------------------------------------------------- append
def check_append(Hq, Hkv, P, new, old, rotary, interleaved, ms, seed, base=10000.0, pad_rows=0):
    rng = np.random.default_rng(seed)
    lens = i32([n + o for n, o in zip(new, old)])
    start = i32(np.concatenate([[0], np.cumsum(new)]))
    T = int(start[-1]) + pad_rows
    table, pages = paged(lens, P, rng, first=old)
    codes, scales = random_cache(pages, Hkv, P, rng)
    qkv = rng.standard_normal((T, Hq + 2 * Hkv, 128))
    qkv[..., rng.choice(128, 5, replace=False)] *= 10
    qkv = qkv.astype(np.float16)
    f = (base ** (-np.arange(0, rotary, 2) / max(rotary, 1))).astype(np.float32)
    gc, gs = dev(codes), dev(scales)
    q0 = torch.full((T, Hq, 128), 7.0, dtype=torch.float16, device=DEV)
    single = max(new) == 1 and min(new) == 1 and not pad_rows
    q = w4a8.kv8_rope_append(dev(qkv.reshape(T, -1)), Hq, gc, gs, dev(table), dev(lens), dev(f),
                             q_start=None if single else dev(start), interleaved=interleaved, rope_scale=ms, out=q0)
    torch.cuda.synchronize()
    assert q.data_ptr() == q0.data_ptr()
    n = int(start[-1])
    pos = np.concatenate([np.arange(o, o + k) for k, o in zip(new, old)])
    x = qkv.astype(np.float64)
    x[:n, :Hq + Hkv] = S.rotate(x[:n, :Hq + Hkv], pos, f, interleaved, ms)
    size = np.abs(qkv.astype(np.float64)).max(axis=2, keepdims=True) * max(ms, 1) * 2
    hq = host(q).astype(np.float64)
    ulp = np.spacing(np.maximum(np.abs(x[:n, :Hq]), 6.2e-5).astype(np.float16)).astype(np.float64)
    assert (np.abs(hq[:n] - x[:n, :Hq]) <= 0.5 * ulp * (1 + 1e-3) + ROT * size[:n, :Hq]).all()
    assert (hq[n:] == 7).all()
    want, sc, written = S.append(x, Hq, codes, scales, table, lens, start)
    hc, hs = host(gc).astype(np.float64), host(gs).astype(np.float64)
    assert (np.abs(hs - sc) <= sc * 4 * ROT).all()
    # with the scale that the kernel wrote taken as given
    want = np.where((written == 1)[..., None], want * (sc / np.maximum(hs, 1e-30))[..., None, None], want)
    off = np.abs(np.clip(want, -127, 127) - hc)
    assert (off[written == 1] <= 0.5 + 127 * 8 * ROT).all(), off[written == 1].max()
    assert (off[written == 2] <= 0.5 + 127 * 4 * ROT).all(), off[written == 2].max()
    untouched = written == 0
    assert np.array_equal(hc[untouched], codes[untouched].astype(np.float64))


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_single_tokens(P, interleaved):
    old = [0, 1, P - 1, P, 2 * P + 5, 1000]
    check_append(8, 2, P, [1] * 6, old, 128, interleaved, 1.0, P)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (12, 4), (5, 1), (32, 8)])
def test_append_ragged_chunks(P, Hq, Hkv):
    check_append(Hq, Hkv, P, [3, 1, 70, 129, 2], [0, 5, P - 1, 64, 1023], 128, False, 1.0, 100 + P + Hq)


@pytest.mark.parametrize("rotary", [0, 2, 50, 64, 96, 126, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_part_of_the_head_and_scaled(rotary, interleaved):
    check_append(4, 2, 32, [40, 9], [0, 37], rotary, interleaved, 1.2773, 200 + rotary)


def test_append_far_positions():
    """Angles of positions up to 2^20, at frequencies near one."""
    check_append(2, 1, 128, [3, 1], [(1 << 20) - 3, 131071], 128, False, 1.0, 300, base=1.5)


def test_append_rows_behind_the_last_sequence_and_empty_sequences():
    check_append(4, 2, 16, [5, 0, 17, 0], [11, 33, 0, 0], 128, False, 1.0, 301, pad_rows=4)


def test_append_many_rows():
    """Past the size from which a block takes several rows of q."""
    check_append(2, 1, 64, [700, 801], [0, 30], 128, True, 1.0, 302)


def test_append_of_zeros_and_a_stale_page():
    """A new page starts from nothing, whatever scale its last owner left; zero vectors give scale 0."""
    codes, scales = w4a8.kv8_cache(2, 1, 16, DEV)
    codes.fill_(99)
    scales.fill_(5.0)
    f, _ = w4a8.rope_frequencies(128, device=DEV)
    table, one = dev(i32([[1]])), dev(i32([1]))
    z = torch.zeros((1, 3 * 128), dtype=torch.float16, device=DEV)
    w4a8.kv8_rope_append(z, 1, codes, scales, table, one, f)
    assert not scales[1].any() and not codes[1, :, :, 0].any()
    assert (codes[1, :, :, 1:] == 99).all() and (scales[0] == 5).all() and (codes[0] == 99).all()
    z[0, 128:] = 2.0  # the second token of the page: zeros carried over to its scale
    w4a8.kv8_rope_append(z, 1, codes, scales, table, one + 1, f)
    assert not codes[1, :, :, 0].any() and (codes[1, 1, :, 1] == 127).all()
    assert torch.equal(scales[1, 1], torch.full((1,), 2.0, device=DEV) / 127)


@pytest.mark.parametrize("P", [16, 64])
def test_append_codes_midway_go_to_the_even_one(P):
    """Values and keys (without rotation: position 0) of a page whose scale is 6 or 14 exactly: x / s is exact
    in 64 bits, many of them midway between two codes."""
    n = P
    v = np.arange(n * 128).reshape(n, 128)
    x = np.zeros((n, 3, 128))
    x[0, 1] = 7 * (v[0] % 255 - 127)   # K, position 0: |x| <= 889, multiples of 7 = s / 2
    x[0, 1, 0] = 14 * 127
    x[:, 2] = 3 * (v % 255 - 127)      # V: multiples of 3 = s / 2, |x| <= 381
    x[0, 2, 0] = 6 * 127
    codes, scales = w4a8.kv8_cache(1, 1, P, DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    f = dev(np.ones(64, np.float32))
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    # the keys' page holds the first token alone, so that no other key sets its scale
    w4a8.kv8_rope_append(dev(x[:1].astype(np.float16)).reshape(1, -1), 1, codes, scales, table, one, f)
    assert scales[0, 0, 0] == 14 and (codes[0, 0, 0, 0].cpu().numpy() == np.rint(x[0, 1] / 14)).all()
    assert scales[0, 1, 0] == 6 and (codes[0, 1, 0, 0].cpu().numpy() == np.rint(x[0, 2] / 6)).all()
    start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    w4a8.kv8_rope_append(dev(x.astype(np.float16)).reshape(n, -1), 1, codes, scales, table, one * n, f, q_start=start)
    assert scales[0, 1, 0] == 6 and (codes[0, 1, 0].cpu().numpy() == np.rint(x[:, 2] / 6)).all()


def test_append_reports_what_it_cannot_place():
    """Lengths beyond the table, pages outside the pool: skipped and reported; the others are placed."""
    codes, scales = w4a8.kv8_cache(4, 1, 16, DEV)
    f, _ = w4a8.rope_frequencies(128, device=DEV)
    x = torch.ones((4, 3 * 128), dtype=torch.float16, device=DEV)
    lens = dev(i32([33, 2, 1, 0]))
    table = dev(i32([[0, 1], [4, 0], [2, 0], [3, 3]]))
    q = torch.full((4, 1, 128), 7.0, dtype=torch.float16, device=DEV)
    w4a8.kv8_rope_append(x, 1, codes, scales, table, lens, f, out=q)
    assert w4a8.get_device_error(DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(DEV)
    assert not codes[0].any() and not codes[1].any() and not codes[3].any() and codes[2, :, :, 0].all()
    assert (q[0] == 7).all() and (q[3] == 7).all() and (q[2] != 7).all()


# ---------------------------------------------------------------- attention
def case(Hq, Hkv, P, new, old, seed, wide=0, pad_rows=0):
    rng = np.random.default_rng(seed)
    lens = i32([n + o for n, o in zip(new, old)])
    start = i32(np.concatenate([[0], np.cumsum(new)]))
    table, pages = paged(lens, P, rng, wide=wide)
    codes, scales = random_cache(pages, Hkv, P, rng)
    q = (rng.standard_normal((int(start[-1]) + pad_rows, Hq, 128)) * 0.5).astype(np.float16)
    return q, codes, scales, table, lens, start


def attend(c, decode, ws=None):
    q, codes, scales, table, lens, start = (dev(a) for a in c)
    y = torch.full_like(q, 7.0)
    if decode:
        w4a8.kv8_attention_decode(q, codes, scales, table, lens, SCALE, out=y, workspace=ws)
    else:
        w4a8.kv8_attention_prefill(q, codes, scales, table, lens, start, SCALE, out=y, workspace=ws)
    torch.cuda.synchronize()
    return host(y)


def check_attention(c, y, weight_eps, heads=None):
    o, E = S.attention(*c, SCALE, weight_eps, heads, 2.0 ** -39 if weight_eps < 2.0 ** -12 else 2.0 ** -35)
    n = int(c[-1][-1])
    hs = slice(None) if heads is None else list(heads)
    o, E, got = o[:n, hs], E[:n, hs], y[:n, hs].astype(np.float64)
    ulp = np.spacing(np.maximum(np.abs(o) + E, 6.2e-5).astype(np.float16)).astype(np.float64)
    assert np.isfinite(got).all()
    bad = np.abs(got - o) / (0.5 * ulp + E)
    assert (bad <= 1).all(), float(bad.max())
    assert (y[n:] == 7).all()


HEADS = [(4, 2), (4, 4), (8, 1), (12, 4), (5, 5), (3, 1), (32, 8), (16, 1), (36, 3)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_decode_within_the_bound(Hq, Hkv, P):
    c = case(Hq, Hkv, P, [1] * 5, [0, 15, 31, 63, 299], 10 * Hq + P)
    check_attention(c, attend(c, True), 2.0 ** -20)


@pytest.mark.parametrize("L", [1, 2, 16, 17, 32, 33, 127, 128, 129, 1000, 5000])
def test_decode_lengths(L):
    c = case(8, 2, 16 if L % 2 else 64, [1], [L - 1], L)
    check_attention(c, attend(c, True), 2.0 ** -20)


def test_decode_many_short_sequences_and_unused_places():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 130)
    lens[[0, 64, 129]] = 0
    c = list(case(4, 2, 16, [1] * 130, [max(int(n) - 1, 0) for n in lens], 6))
    c[4] = i32(lens)
    y = attend(c, True)
    c2 = [c[0], c[1], c[2], c[3], c[4], c[5]]
    check_attention(c2, y, 2.0 ** -20)
    assert not y[[0, 64, 129]].any()


def test_decode_long_and_short_together():
    c = case(8, 1, 32, [1] * 4, [20000, 0, 70, 3999], 7, wide=9)
    check_attention(c, attend(c, True), 2.0 ** -20, heads=(0, 7))


def test_decode_full_size():
    """The heads of the decode workload, 16 sequences of 2048 to 4096 tokens, on sampled heads."""
    wl = I.KV_WORKLOADS["kv-decode"]
    Hq, Hkv, _ = wl.heads
    lens = I.kv_seq_lens(wl, I.seed_of("t-kv8lens"))
    c = case(Hq, Hkv, 64, [1] * wl.batch, [int(n) - 1 for n in lens], 8)
    check_attention(c, attend(c, True), 2.0 ** -20, heads=(0, 13, 31))


@pytest.mark.parametrize("decode", [True, False])
def test_attention_does_not_look_behind_the_end(decode):
    """Codes behind a sequence's end, pages of nobody, table entries behind the end and their scales do not matter."""
    new = [1, 1, 1] if decode else [3, 20, 1]
    c = list(case(8, 2, 32, new, [40, 99, 0], 9, wide=3))
    y1 = attend(c, decode)
    q, codes, scales, table, lens, start = c
    used = np.zeros(codes.shape[:1] + codes.shape[3:4], bool)
    for b in range(3):
        for p in range(int(lens[b])):
            used[table[b, p // 32], p % 32] = True
    codes = np.where(used[:, None, None, :, None], codes, np.int8(-128))
    scales = np.where(used.any(1)[:, None, None], scales, np.float32(np.nan))
    table = np.where(np.arange(table.shape[1]) < -(-lens[:, None] // 32), table, 1 << 30).astype(np.int32)
    y2 = attend([q, codes, scales, table, lens, start], decode)
    assert np.array_equal(y1.view(np.uint16), y2.view(np.uint16))


@pytest.mark.parametrize("decode", [True, False])
def test_attention_extreme_scores_and_scales(decode):
    """Scores far apart (one token takes all), scales 0, tiny and large in neighbouring pages."""
    new = [1, 1] if decode else [4, 33]
    c = list(case(8, 2, 16, new, [95, 300], 11))
    rng = np.random.default_rng(12)
    c[0] = (rng.standard_normal(c[0].shape) * 40).astype(np.float16)
    c[2] = rng.choice(np.float32([0.0, 1e-7, 1e-3, 1.0, 100.0]), c[2].shape).astype(np.float32)
    c[2][:, 0] = np.minimum(c[2][:, 0], np.float32(0.05))
    check_attention(c, attend(c, decode), 2.0 ** (-20 if decode else -11))


@pytest.mark.parametrize("decode", [True, False])
def test_attention_of_all_zero_values(decode):
    c = list(case(4, 1, 16, [1, 1] if decode else [2, 9], [10, 40], 13))
    c[2] = np.zeros_like(c[2])
    assert not attend(c, decode)[:int(c[5][-1])].any()


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("P", [16, 64, 128])
def test_prefill_within_the_bound(Hq, Hkv, P):
    c = case(Hq, Hkv, P, [1, 5, 40, 0, 17], [0, 100, 0, 9, 333], 20 * Hq + P, pad_rows=3)
    check_attention(c, attend(c, False), 2.0 ** -11)


@pytest.mark.parametrize("n,old", [(1, 0), (2, 1), (31, 0), (33, 31), (64, 64), (127, 1), (128, 0), (129, 128), (257, 3),
                                   (300, 1000), (1, 2000), (7, 4000)])
def test_prefill_lengths(n, old):
    c = case(4, 1, 32, [n], [old], 1000 + n)
    check_attention(c, attend(c, False), 2.0 ** -11, heads=(0, 3))


def test_prefill_many_sequences():
    rng = np.random.default_rng(21)
    new, old = rng.integers(0, 12, 90), rng.integers(0, 200, 90)
    c = case(6, 2, 16, [int(n) for n in new], [int(n) for n in old], 22)
    check_attention(c, attend(c, False), 2.0 ** -11)


@pytest.mark.parametrize("Hq,Hkv,n,old", [(4, 1, 300, 5000), (8, 8, 260, 3000), (32, 2, 130, 1500), (3, 1, 1000, 500)])
def test_prefill_cut_into_parts(Hq, Hkv, n, old):
    """A chunk over a long context: each piece of 256 rows cut over many CTAs and joined; an odd
    group, rows behind the sequence, a workspace full of garbage behind its counters."""
    c = case(Hq, Hkv, 32, [n, 0, 19], [old, 40, 700], 500 + n, pad_rows=3)
    ws = torch.full((w4a8.kv8_workspace_bytes(3, n + 22, Hq, Hkv),), 0x7F, dtype=torch.uint8, device=DEV)
    ws[:4096] = 0
    y = attend(c, False, ws)
    check_attention(c, y, 2.0 ** -11, heads=(0, Hq - 1))
    assert np.array_equal(y.view(np.uint16), attend(c, False, ws).view(np.uint16))


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (32, 8), (6, 6), (12, 1)])
def test_prefill_few_and_many_rows_together(Hq, Hkv):
    """Sequences of a few rows beside long chunks, ragged limits that end a tile early, padding rows behind."""
    c = case(Hq, Hkv, 32, [1, 300, 8, 2, 0, 9, 33, 5], [500, 70, 0, 31, 7, 1000, 95, 3000], 400 + Hq, pad_rows=5)
    check_attention(c, attend(c, False), 2.0 ** -11)


def test_prefill_one_sequence_with_padding_rows():
    """More rows in the batch than the one sequence has."""
    c = case(4, 1, 16, [3], [50], 24, pad_rows=200)
    check_attention(c, attend(c, False), 2.0 ** -11)


def test_prefill_of_single_tokens_is_decode():
    c = case(8, 2, 64, [1] * 6, [0, 64, 700, 5, 63, 200], 23)
    check_attention(c, attend(c, False), 2.0 ** -11)


def test_attention_repeats_bit_for_bit_and_leaves_the_workspace_clean():
    c = case(32, 8, 64, [1] * 4, [3000, 1, 700, 1023], 24)
    g = [dev(a) for a in c]
    ws = torch.zeros(max(w4a8.kv8_workspace_bytes(4, 4, 32, 8), w4a8.kv8_workspace_bytes(3, 247, 8, 2)),
                     dtype=torch.uint8, device=DEV)
    ref = dev(attend(c, True, ws)).view(torch.int16)
    out = torch.empty_like(g[0])
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(300):
        w4a8.kv8_attention_decode(*g[:5], SCALE, out=out, workspace=ws)
        bad += (out.view(torch.int16) != ref).any()
    assert int(bad) == 0
    c = case(8, 2, 64, [40, 7, 200], [300, 1000, 0], 25)
    g = [dev(a) for a in c]
    ref = dev(attend(c, False, ws)).view(torch.int16)
    out = torch.empty_like(g[0])
    for _ in range(100):
        w4a8.kv8_attention_prefill(*g, SCALE, out=out, workspace=ws)
        bad += (out.view(torch.int16) != ref).any()
    assert int(bad) == 0


def test_attention_output_in_place_of_the_query():
    for c, decode in ((case(8, 2, 64, [1] * 3, [3000, 0, 700], 33), True), (case(8, 2, 64, [5, 300], [3000, 20], 34), False)):
        ref = attend(c, decode)
        g = [dev(a) for a in c]
        if decode:
            w4a8.kv8_attention_decode(*g[:5], SCALE, out=g[0])
        else:
            w4a8.kv8_attention_prefill(*g, SCALE, out=g[0])
        assert np.array_equal(host(g[0]).view(np.uint16), ref.view(np.uint16))


def test_attention_with_a_negative_and_a_zero_scale():
    """Softmax of the negated scores; every token alike."""
    for decode in (True, False):
        c = case(8, 2, 32, [1, 1] if decode else [40, 3], [100, 20], 35)
        g = [dev(a) for a in c]
        call = (lambda s: w4a8.kv8_attention_decode(*g[:5], s)) if decode else (lambda s: w4a8.kv8_attention_prefill(*g, s))
        y = host(call(-SCALE))
        o, E = S.attention(*c, -SCALE, 2.0 ** -11, None, 2.0 ** -35)
        ulp = np.spacing(np.maximum(np.abs(o) + E, 6.2e-5).astype(np.float16)).astype(np.float64)
        assert (np.abs(y.astype(np.float64) - o) <= 0.5 * ulp + E).all()
        y = host(call(0.0))
        o, E = S.attention(*c, 0.0, 2.0 ** -11, None, 2.0 ** -35)
        ulp = np.spacing(np.maximum(np.abs(o) + E, 6.2e-5).astype(np.float16)).astype(np.float64)
        assert (np.abs(y.astype(np.float64) - o) <= 0.5 * ulp + E).all()


def test_shared_pages_between_sequences():
    """A common prefix held once: several tables name the same pages."""
    for decode in (True, False):
        c = list(case(8, 2, 32, [1, 1, 1] if decode else [30, 40, 2], [200, 230, 300], 36))
        c[3] = c[3].copy()
        c[3][1:, :6] = c[3][0, :6]
        check_attention(c, attend(c, decode), 2.0 ** (-20 if decode else -11))


def test_starts_that_fall_are_reported_and_stay_in_bounds():
    c = list(case(4, 2, 16, [5, 9, 7], [20, 30, 40], 37))
    c[5] = i32([0, 14, 5, 21])
    g = [dev(a) for a in c]
    w4a8.kv8_attention_prefill(*g, SCALE)
    assert w4a8.get_device_error(DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(DEV)
    f, _ = w4a8.rope_frequencies(128, device=DEV)
    qkv = torch.zeros((21, 8 * 128), dtype=torch.float16, device=DEV)
    w4a8.kv8_rope_append(qkv, 4, g[1], g[2], g[3], g[4], f, q_start=dev(i32([-7, 14, 5, 1 << 30])))
    assert w4a8.get_device_error(DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(DEV)


def test_prefill_in_a_graph_with_other_lengths():
    c = case(8, 2, 64, [40, 300, 3], [3000, 20, 100], 38)
    g = [dev(a) for a in c]
    out = torch.empty_like(g[0])
    w4a8.kv8_attention_prefill(*g, SCALE, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4a8.kv8_attention_prefill(*g, SCALE, out=out)
    new, old = [300, 3, 40], [20, 2900, 0]
    start, lens = i32(np.concatenate([[0], np.cumsum(new)])), i32([n + o for n, o in zip(new, old)])
    table = c[3].copy()
    table[0], table[1] = c[3][1], c[3][0]
    for t, a in zip(g[3:], (table, lens, start)):
        t.copy_(dev(a))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check_attention((c[0], c[1], c[2], table, lens, start), host(out), 2.0 ** -11, heads=(0, 5))


def test_two_streams_at_once_without_a_workspace():
    """The binding keeps a workspace per stream: calls on two streams may overlap."""
    cs = [case(8, 2, 64, [1] * 3, [3000, 900, 2000], s) for s in (26, 27)]
    refs = [dev(attend(c, True)) for c in cs]
    gs = [[dev(a) for a in c[:5]] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(50):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[k].append(w4a8.kv8_attention_decode(*gs[k], SCALE))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(o, refs[k]) for o in outs[k])


def test_two_graphs_with_their_own_workspaces():
    """Two captured calls replayed on two streams at once, lengths changed between replays."""
    cs = [case(8, 2, 64, [1] * 3, [3000, 900, 2000], s) for s in (28, 29)]
    gs = [[dev(a) for a in c[:5]] for c in cs]
    outs = [torch.empty_like(g[0]) for g in gs]
    graphs = []
    for g, o in zip(gs, outs):
        w4a8.kv8_attention_decode(*g, SCALE, out=o)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w4a8.kv8_attention_decode(*g, SCALE, out=o)
        graphs.append(graph)
    shorter = i32([130, 1, 2001])
    for g in gs:
        g[4].copy_(dev(shorter))
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(30):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        check_attention(c[:4] + (shorter, c[5]), host(o), 2.0 ** -20)


def test_attention_reports_bad_lengths_and_pages():
    """No access leaves the buffers; the other sequences keep their values."""
    c = list(case(4, 2, 16, [1] * 4, [20, 30, 40, 9], 30))
    ref = attend(c, True)
    c[4] = c[4].copy()
    c[3] = c[3].copy()
    c[4][0], c[3][1, 1] = 1 << 20, 1 << 29
    y = attend(c, True)
    assert w4a8.get_device_error(DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(DEV)
    assert np.array_equal(y[2:], ref[2:])
    c = list(case(4, 2, 16, [2, 3, 4], [20, 30, 40], 31))
    ref = attend(c, False)
    c[4], c[3] = c[4].copy(), c[3].copy()
    c[4][0], c[3][1, 0] = 1, -5
    y = attend(c, False)
    assert w4a8.get_device_error(DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(DEV)
    assert np.array_equal(y[5:], ref[5:])


def test_kv8_refuses_mismatched_tensors():
    q, codes, scales, table, lens, start = (dev(a) for a in case(4, 2, 16, [1, 1], [20, 30], 32))
    ok = dict(q=q, kv_codes=codes, kv_scales=scales, block_table=table, seq_lens=lens, scale=SCALE)
    for kw in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[..., :64]), dict(kv_codes=codes.view(torch.uint8)),
               dict(kv_codes=codes[0]), dict(kv_scales=scales[:1]), dict(kv_scales=scales.half()),
               dict(block_table=table.long()), dict(block_table=table[:1]), dict(seq_lens=lens.long()),
               dict(seq_lens=lens[:1]), dict(out=q.float()), dict(out=q[:1]), dict(seq_lens=lens.cpu()),
               dict(workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)), dict(workspace=q)):
        with pytest.raises(w4a8.W4A8Error):
            w4a8.kv8_attention_decode(**{**ok, **kw})
    for bad in (start.long(), start[:2], start.cpu()):
        with pytest.raises(w4a8.W4A8Error):
            w4a8.kv8_attention_prefill(q, codes, scales, table, lens, bad, SCALE)


# --------------------------------------------------------- the run together
def test_a_layer_as_it_is_used():
    """norm -> GEMM (q, k, v) -> rotation and append -> attention: a prompt in two
    chunks, then single tokens, each stage checked from what the last one gave."""
    Hq, Hkv, P, K = 4, 2, 16, 256
    N = (Hq + 2 * Hkv) * 128
    rng = np.random.default_rng(40)
    codes, scales = w4a8.kv8_cache(24, Hkv, P, DEV)
    table = dev(i32(rng.permutation(24).reshape(2, 12)))
    f, ms = w4a8.rope_frequencies(64, 10000.0, "ramp", 4.0, 64, device=DEV)
    wcodes = list(I.uniform_codes(N, K, 41))
    blob = w4a8.pack_weights(*(dev(c) for c in wcodes))
    weight = dev((1 + 0.1 * rng.standard_normal(K)).astype(np.float16))
    done = [0, 0]
    hk = np.zeros(codes.shape, np.int8)
    hs = np.zeros(scales.shape, np.float32)
    for new in ([30, 17], [25, 60], [1, 1], [1, 1], [0, 1], [1, 1]):
        T = sum(new)
        x, r = (dev(I.activations(T, K, 42 + done[0] + k)) for k in (0, 1))
        h, A8, sA, rs = w4a8.rmsnorm_quantize_act(x, weight, 1e-5, residual=r)
        qkv = w4a8.gemm(A8, sA, rs, blob, N, K)
        old = list(done)
        done = [a + b for a, b in zip(done, new)]
        lens, start = i32(done), i32([0, new[0], T])
        single = new == [1, 1]
        q = w4a8.kv8_rope_append(qkv, Hq, codes, scales, table, dev(lens), f, q_start=None if single else dev(start),
                                 rope_scale=ms)
        if single:
            y = w4a8.kv8_attention_decode(q, codes, scales, table, dev(lens), SCALE * 0.05)
        else:
            y = w4a8.kv8_attention_prefill(q, codes, scales, table, dev(lens), dev(start), SCALE * 0.05)
        torch.cuda.synchronize()
        rot = host(qkv).reshape(T, -1, 128).astype(np.float64)
        pos = np.concatenate([np.arange(o, o + n) for o, n in zip(old, new)])
        rot[:, :Hq + Hkv] = S.rotate(rot[:, :Hq + Hkv], pos, host(f), False, ms)
        want, sc, written = S.append(rot, Hq, hk, hs, host(table), lens, start)
        hk, hs = host(codes).copy(), host(scales).copy()
        assert (np.abs(hs - sc) <= sc * 8 * ROT).all()
        assert (np.abs(np.clip(want, -127, 127) - hk)[written > 0] <= 0.5 + 127 * 16 * ROT).all()
        o, E = S.attention(host(q), hk, hs, host(table), lens, start, SCALE * 0.05, 2.0 ** -11)
        ulp = np.spacing(np.maximum(np.abs(o) + E, 6.2e-5).astype(np.float16)).astype(np.float64)
        assert (np.abs(host(y).astype(np.float64) - o) <= 0.5 * ulp + E).all()
