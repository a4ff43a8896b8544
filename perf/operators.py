"""The serving operators around the W4A8 GEMMs, as cases to be measured.

Four operators of a decoder layer whose linears are W4A8 GEMMs:

* ``norm``    residual addition, root-mean-square norm, int8 codes with a scale per token (what the GEMM takes)
* ``append``  rotary positions for q and k, k and v quantized into a paged cache of int8 codes with a scale per (page, head)
* ``decode``  attention of one new token per sequence over that cache
* ``prefill`` causal attention of many new tokens per sequence over that cache, which already holds them

Cache: codes int8 [pages, 2 (K, V), kv heads, page, 128], scales fp32 [pages, 2, kv heads]; a sequence's tokens lie in the pages that its
row of the block table names. Codes are returned as the values that they stand for, in fp16.
"""
import math
import random

import torch

own = False

DEV = "cuda"
D = 128
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of a decode step's first GEMM, one user: latency
        {"name": "norm_1x4096", "op": "norm", "rows": 1, "width": 4096, "residual": True},
        # the norm of a mixed batch of prompts, an odd number of tokens and a width that no power of two divides, no residual yet
        {"name": "norm_1237x7176", "op": "norm", "rows": 1237, "width": 7176, "residual": False},
        # the norm of a full prefill batch: bandwidth
        {"name": "norm_8192x4096", "op": "norm", "rows": 8192, "width": 4096, "residual": True},
        # one decode step of 16 users: each appends a token in the middle of a page
        {"name": "append_16x1", "op": "append", "batch": 16, "new_lo": 1, "new_hi": 1, "old_lo": 2047, "old_hi": 4095, "heads": 32,
         "kv_heads": 8, "page": 64, "rotary": 128, "interleaved": False, "scaling": "none"},
        # chunks of a few prompts that go on in pages begun before, part of the head rotated, neighbours paired
        {"name": "append_5x300", "op": "append", "batch": 5, "new_lo": 37, "new_hi": 611, "old_lo": 0, "old_hi": 130001, "heads": 12,
         "kv_heads": 4, "page": 16, "rotary": 64, "interleaved": True, "scaling": "linear"},
        # a prefill batch of new prompts
        {"name": "append_4x2048", "op": "append", "batch": 4, "new_lo": 1900, "new_hi": 2196, "old_lo": 0, "old_hi": 0, "heads": 32,
         "kv_heads": 8, "page": 64, "rotary": 128, "interleaved": False, "scaling": "bands"},
        # one user, a short context: latency
        {"name": "decode_1x500", "op": "decode", "batch": 1, "len_lo": 500, "len_hi": 500, "heads": 32, "kv_heads": 8, "page": 64},
        # 16 users with 2048 to 4096 cached tokens
        {"name": "decode_16x4096", "op": "decode", "batch": 16, "len_lo": 2048, "len_hi": 4096, "heads": 32, "kv_heads": 8, "page": 64},
        # 8 users, no shared heads: the most cache for each query
        {"name": "decode_8x4096_mha", "op": "decode", "batch": 8, "len_lo": 2048, "len_hi": 4096, "heads": 64, "kv_heads": 64, "page": 64},
        # a batch of new prompts, ragged
        {"name": "prefill_3x2048", "op": "prefill", "batch": 3, "new_lo": 1500, "new_hi": 2100, "old_lo": 0, "old_hi": 0, "heads": 32,
         "kv_heads": 8, "page": 64},
        # a chunk of one long prompt: 1000 new tokens over what came before
        {"name": "prefill_1000_of_9000", "op": "prefill", "batch": 1, "new_lo": 1000, "new_hi": 1000, "old_lo": 8017, "old_hi": 8017,
         "heads": 32, "kv_heads": 8, "page": 16},
        # guesses of a small model to be checked: a handful of tokens for each user
        {"name": "prefill_8x5", "op": "prefill", "batch": 8, "new_lo": 3, "new_hi": 6, "old_lo": 900, "old_hi": 2500, "heads": 32,
         "kv_heads": 8, "page": 64},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 8), (64, 64), (64, 8), (8, 2), (12, 4), (8, 1), (5, 5), (4, 2), (48, 3))


def draw(rng):
    op = rng.choice(("norm", "append", "decode", "prefill"))
    if op == "norm":
        width = 8 * _log(rng, 8, 3500)
        return {"op": op, "rows": _log(rng, 1, max(1, min(8192, (1 << 25) // width))), "width": width,
                "residual": rng.random() < 0.7}
    heads, kv = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        batch = _log(rng, 1, 64)
        most = max(1, 6000 * 48 // ((heads + 2 * kv) * batch))
        new = 1 if rng.random() < 0.3 else _log(rng, 1, most)
        old = rng.choice((0, _log(rng, 1, 30000)))
        rotary = rng.choice((128, 128, 64, 32, 50, 2))
        return {"op": op, "batch": batch, "new_lo": max(1, new // 2), "new_hi": new, "old_lo": old // 3, "old_hi": old, "heads": heads,
                "kv_heads": kv, "page": page, "rotary": rotary, "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(("none", "linear", "bands", "ramp"))}
    if op == "decode":
        batch = _log(rng, 1, 64)
        most = _log(rng, 1, max(1, 40 * 4096 * 8 // (batch * kv)))
        return {"op": op, "batch": batch, "len_lo": rng.choice((1, (most + 1) // 2, most)), "len_hi": most, "heads": heads,
                "kv_heads": kv, "page": page}
    batch = _log(rng, 1, 12)
    old = rng.choice((0, _log(rng, 1, 9000 // batch)))
    pairs = 220_000_000 // (heads * batch)  # of each head and sequence
    new = _log(rng, 1, max(1, int(math.sqrt(old * old + 2 * pairs) - old)))
    return {"op": op, "batch": batch, "new_lo": max(1, new // 2), "new_hi": new, "old_lo": old // 3, "old_hi": old, "heads": heads,
            "kv_heads": kv, "page": page}


def _spread(lo, hi, n, what):
    """n whole numbers between lo and hi, the largest among them, the same ones every time."""
    r = random.Random("%s %d %d %d" % (what, lo, hi, n))
    got = [r.randint(lo, hi) for _ in range(n)]
    got[r.randrange(n)] = hi
    return got


def _lengths(case):
    """(new tokens, tokens cached before the call) of each sequence."""
    n = case["batch"]
    if case["op"] == "decode":
        return [1] * n, [x - 1 for x in _spread(case["len_lo"], case["len_hi"], n, "len")]
    return _spread(case["new_lo"], case["new_hi"], n, "new"), _spread(case["old_lo"], case["old_hi"], n, "old")


def work(case):
    if case["op"] == "norm":
        M, K = case["rows"], case["width"]
        return {"bytes": M * K * (7 if case["residual"] else 3) + 2 * K + 6 * M, "flops": 8 * M * K}
    Hq, Hkv, P = case["heads"], case["kv_heads"], case["page"]
    new, old = _lengths(case)
    T = sum(new)
    if case["op"] == "append":
        # the rows of q, k and v in, q and the codes out, the scales of the pages written
        pages = sum((o + n - 1) // P - o // P + 1 for n, o in zip(new, old))
        return {"bytes": T * (Hq + 2 * Hkv) * 2 * D + T * Hq * 2 * D + T * 2 * Hkv * D + pages * 2 * Hkv * 4, "flops": 10 * T * (Hq + 2 * Hkv) * D}
    cached = sum(n + o for n, o in zip(new, old))
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    pages = sum(-(-(n + o) // P) for n, o in zip(new, old))
    return {"bytes": cached * Hkv * 2 * D + pages * (2 * Hkv * 4 + 4) + 4 * T * Hq * D, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ inputs
def _frequencies(rotary, scaling):
    """Rotation per position (fp32, one for each pair) and the factor on the rotated values, worked out once by a user's program."""
    i = torch.arange(0, rotary, 2, dtype=torch.float64)
    f = 500000.0 ** (-i / rotary)
    if scaling == "none":
        return f.float(), 1.0
    if scaling == "linear":  # positions stretched by 8
        return (f / 8).float(), 1.0
    old = 8192.0
    if scaling == "bands":  # slow rotations stretched, fast ones kept, those between blended
        low, high, factor = 1.0, 4.0, 8.0
        t = ((old * f / (2 * math.pi)) - low) / (high - low)
        t = t.clamp(0, 1)
        return ((1 - t) * f / factor + t * f).float(), 1.0
    # a ramp over the pair's index between those that turn 32 times and once within the old length, values scaled
    factor = 16.0
    at = lambda turns: rotary * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(500000.0))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rotary - 1)
    t = ((torch.arange(rotary // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return (t * f / factor + (1 - t) * f).float(), 0.1 * math.log(factor) + 1


def _outliers(width, share, factor):
    """A factor for each channel: a few channels of real activations are much larger than the rest, the same ones for every token."""
    g = torch.Generator().manual_seed(width)
    f = torch.ones(width)
    f[torch.randperm(width, generator=g)[: int(share * width + 0.5)]] = factor
    return f.to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    if case["op"] == "norm":
        M, K = case["rows"], case["width"]
        out = _outliers(K, 0.01, 20.0)
        s = {"op": "norm", "x": (normal(M, K) * out).half(), "w": (1 + 0.1 * normal(K)).half(),
             "r": (normal(M, K) * out).half() if case["residual"] else None}
        s["sum"] = torch.empty(M, dtype=torch.float16, device=DEV)
        s["out"] = (torch.empty_like(s["x"]) if case["residual"] else None, torch.empty(M, K, dtype=torch.int8, device=DEV),
                    torch.empty(M, dtype=torch.float16, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV))
        return s
    B, Hq, Hkv, P = case["batch"], case["heads"], case["kv_heads"], case["page"]
    new, old = _lengths(case)
    T = sum(new)
    lens = [n + o for n, o in zip(new, old)]
    wide = -(-max(lens) // P)
    # the pages that the call touches come first in the pool, the others in any order behind them
    touched, rest, table = [], [], torch.zeros(B, wide, dtype=torch.int64)
    for b in range(B):
        first = old[b] // P if case["op"] == "append" else 0
        for p in range(-(-lens[b] // P)):
            (touched if p >= first else rest).append((b, p))
    if case["op"] == "append":
        rest = rest[:64]  # pages that an append does not look at: a few are enough
    order = torch.randperm(len(touched), generator=torch.Generator().manual_seed(int(seed))).tolist()
    for at, (b, p) in zip(order, touched):
        table[b, p] = at
    for at, (b, p) in enumerate(rest):
        table[b, p] = len(touched) + at
    pages = len(touched) + len(rest)
    outk = _outliers(D, 0.04, 10.0)
    codes = torch.empty(pages, 2, Hkv, P, D, dtype=torch.int8, device=DEV)
    scales = torch.empty(pages, 2, Hkv, device=DEV)
    for i in range(0, pages, 1024):  # in pieces: the largest caches are long
        x = normal(min(1024, pages - i), 2, Hkv, P, D)
        x[:, 0] *= outk
        sc = x.abs().amax((3, 4)) / 127
        codes[i:i + 1024] = (x / sc[..., None, None]).round().clamp(-127, 127).to(torch.int8)
        scales[i:i + 1024] = sc
    s = {"op": case["op"], "codes": codes, "scales": scales, "table": table.to(torch.int32).to(DEV), "T": T, "P": P, "Hq": Hq, "Hkv": Hkv,
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "scale": 1 / math.sqrt(D)}
    s["start"] = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    s["single"] = max(new) == 1 and min(new) == 1
    # host facts of the batch, as a scheduler has them: of each new token its sequence and position
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    pos = torch.cat([torch.arange(o, o + n) for n, o in zip(new, old)])
    s["seq"], s["pos"], s["most"] = seq.to(DEV), pos.to(DEV), max(new)
    if case["op"] == "append":
        f, ms = _frequencies(case["rotary"], case["scaling"])
        s |= {"inv_freq": f.to(DEV), "ms": ms, "interleaved": case["interleaved"], "rotary": case["rotary"], "touched": len(touched)}
        x = normal(T, Hq + 2 * Hkv, D)
        x[:, :Hq + Hkv] *= outk
        s["qkv"] = x.view(T, -1).half()
        # the touched pages, in the pool's order: sequence, number within the sequence
        by = sorted(zip(order, touched))
        s["page_seq"] = torch.tensor([b for _, (b, _) in by], device=DEV)
        s["page_no"] = torch.tensor([p for _, (_, p) in by], device=DEV)
        s["old"] = torch.tensor(old, device=DEV)
        s["q"] = torch.empty(T, Hq, D, dtype=torch.float16, device=DEV)
        s["values"] = torch.empty(len(touched), 2, Hkv, P, D, dtype=torch.float16, device=DEV)
        s["touched_codes"], s["touched_scales"] = codes[:len(touched)], scales[:len(touched), :, :, None, None]
        # pages that the call begins hold nothing yet; in the others nothing lies behind the tokens cached before
        n_old = (s["old"][s["page_seq"]] - s["page_no"] * P).clamp(min=0)
        codes[:len(touched)] *= (torch.arange(P, device=DEV) < n_old[:, None])[:, None, None, :, None]
        scales[:len(touched)] *= (n_old > 0)[:, None, None]
    else:
        s["q"] = (normal(T, Hq, D)).half()
        s["y"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"norm": _norm, "append": _append, "decode": _attention, "prefill": _attention}[state["op"]](state)


def _norm(s):
    if own:
        import w4a8_quantized_gemm_quantize_b200 as w4a8
        h, codes, sA, rowsum = w4a8.rmsnorm_quantize_act(s["x"], s["w"], EPS, residual=s["r"], out=s["out"])
    else:
        h = None if s["r"] is None else (s["x"].float() + s["r"].float()).half()
        v = (s["x"] if h is None else h).float()
        y = v * (1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)) * s["w"].float()
        sA = (y.abs().amax(1) / 127).half()
        sf = sA.float()[:, None]
        codes = torch.where(sf > 0, (y / torch.where(sf > 0, sf, 1)).round().clamp(-127, 127), 0).to(torch.int8)
        rowsum = codes.sum(1, dtype=torch.int32)
    # codes as the values that they stand for, their sum in units of the largest code
    return {"h": h, "a": torch.mul(codes, sA[:, None]), "scale": sA, "sum": torch.mul(rowsum, 1 / 127, out=s["sum"])}


def _rotate(x, cos, sin, interleaved, rotary):
    """x [T, heads, 128] in 32 bits, the first `rotary` values of each head rotated."""
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rotary // 2], r[..., rotary // 2:])
    u, v = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((r, x[..., rotary:]), -1)


def _append(s):
    Hq, Hkv, P, n = s["Hq"], s["Hkv"], s["P"], s["touched"]
    if own:
        import w4a8_quantized_gemm_quantize_b200 as w4a8
        q = w4a8.kv8_rope_append(s["qkv"], Hq, s["codes"], s["scales"], s["table"], s["lens"], s["inv_freq"],
                                 q_start=None if s["single"] else s["start"], interleaved=s["interleaved"], rope_scale=s["ms"], out=s["q"])
    else:
        x = s["qkv"].view(s["T"], Hq + 2 * Hkv, D).float()
        angle = (s["pos"].double()[:, None] * s["inv_freq"].double())[:, None]
        cos, sin = (angle.cos() * s["ms"]).float(), (angle.sin() * s["ms"]).float()
        x[:, :Hq + Hkv] = _rotate(x[:, :Hq + Hkv], cos, sin, s["interleaved"], s["rotary"])
        q = x[:, :Hq].half()
        # the touched pages: for each of their places the new token that goes there, or none
        at = s["page_no"][:, None] * P + torch.arange(P, device=DEV)
        old = s["old"][s["page_seq"]][:, None]
        is_new = (at >= old) & (at < s["lens"][s["page_seq"]][:, None])
        token = torch.where(is_new, s["start"][s["page_seq"]][:, None] + at - old, 0)
        v = x[:, Hq:].view(s["T"], 2, Hkv, D)[token].permute(0, 2, 3, 1, 4) * is_new[:, None, None, :, None]
        before = s["scales"][:n] * (s["page_no"] * P < old[:, 0])[:, None, None]
        after = torch.maximum(before, v.abs().amax((3, 4)) / 127)
        by = torch.where(after > 0, after, 1)[..., None, None]
        kept = (s["codes"][:n].float() * (before / after.clamp(min=1e-38))[..., None, None]).round()
        fresh = (v / by).round().clamp(-127, 127)
        s["codes"][:n] = torch.where(is_new[:, None, None, :, None], fresh, kept).to(torch.int8)
        s["scales"][:n] = after
    # the touched pages as the values that they stand for
    torch.mul(s["touched_codes"], s["touched_scales"], out=s["values"])
    return {"q": q, "kv": s["values"]}


def _attention(s):
    if own:
        import w4a8_quantized_gemm_quantize_b200 as w4a8
        if s["op"] == "decode":
            return w4a8.kv8_attention_decode(s["q"], s["codes"], s["scales"], s["table"], s["lens"], s["scale"], out=s["y"])
        return w4a8.kv8_attention_prefill(s["q"], s["codes"], s["scales"], s["table"], s["lens"], s["start"], s["scale"], out=s["y"])
    B, Hq, Hkv = len(s["lens"]), s["Hq"], s["Hkv"]
    table = s["table"].long()
    kv = s["codes"][table].float() * s["scales"][table][..., None, None]  # [B, blocks, 2, Hkv, page, 128]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hkv, -1, D)
    n, G = s["most"], Hq // Hkv
    row = s["pos"] - (s["lens"] - (s["start"][1:] - s["start"][:-1]))[s["seq"]]  # of each new token its number within the call
    q = torch.zeros(B, n, Hq, D, device=DEV)
    q[s["seq"], row] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    z = torch.matmul(q, kv[0].transpose(2, 3)) * s["scale"]
    first = s["lens"] - (s["start"][1:] - s["start"][:-1])
    sees = torch.arange(kv.shape[3], device=DEV) <= (first[:, None] + torch.arange(n, device=DEV))[..., None]
    z = z.view(B, Hkv, G, n, -1).masked_fill_(~sees[:, None, None], -math.inf)
    z = torch.exp(z - z.amax(4, keepdim=True))
    z = (z / z.sum(4, keepdim=True)).view(B, Hkv, G * n, -1)
    y = torch.matmul(z, kv[1]).view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return y[s["seq"], row].half()


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double()
        h = None
        if s["r"] is not None:
            h = v + s["r"].double()
            v = h.half().double()
        y = v / ((v ** 2).sum(1, keepdim=True) / case["width"] + EPS).sqrt() * s["w"].double()
        sA = (y.abs().amax(1) / 127).half().double()
        codes = (y / sA[:, None].clamp(min=1e-30)).round().clamp(-127, 127)
        return {"h": h, "a": codes * sA[:, None], "scale": y.abs().amax(1) / 127, "sum": codes.sum(1) / 127}
    Hq, Hkv, P = s["Hq"], s["Hkv"], s["P"]
    new, old = _lengths(case)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    if case["op"] == "append":
        x = s["qkv"].double().view(s["T"], -1, D)
        half = case["rotary"] // 2
        pair = torch.arange(half, device=DEV)
        ia, ib = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
        t = torch.polar(torch.full((s["T"], half), float(s["ms"]), dtype=torch.float64, device=DEV),
                        s["pos"].double()[:, None] * s["inv_freq"].double()[None])
        turned = torch.complex(x[:, :Hq + Hkv, ia], x[:, :Hq + Hkv, ib]) * t[:, None]
        x[:, :Hq + Hkv, ia], x[:, :Hq + Hkv, ib] = turned.real, turned.imag
        values = torch.zeros(s["touched"], 2, Hkv, P, D, dtype=torch.float64, device=DEV)
        table = s["table"].cpu().tolist()
        for b in range(case["batch"]):
            for p in range(old[b] // P, -(-(old[b] + new[b]) // P)):
                at = table[b][p]
                lo, hi = max(old[b], p * P), min(old[b] + new[b], (p + 1) * P)
                v = x[starts[b] + lo - old[b]:starts[b] + hi - old[b], Hq:].view(hi - lo, 2, Hkv, D).permute(1, 2, 0, 3)
                after = v.abs().amax((2, 3)) / 127
                if lo > p * P:
                    before = s["scales"][at].double()
                    after = torch.maximum(after, before)
                    kept = s["codes"][at, :, :, :lo - p * P].double() * (before / after)[..., None, None]
                    values[at, :, :, :lo - p * P] = kept.round() * after[..., None, None]
                values[at, :, :, lo - p * P:hi - p * P] = (v / after[..., None, None]).round() * after[..., None, None]
        return {"q": x[:, :Hq], "kv": values}
    pairs = sum(n * (n + o) for n, o in zip(new, old)) * Hq
    if pairs > 3e10:
        return None
    y = torch.empty(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    for b in range(case["batch"]):
        n, L = new[b], new[b] + old[b]
        rows = s["table"][b, :-(-L // P)].long()
        for h in range(Hkv):
            kv = (s["codes"][rows, :, h].double() * s["scales"][rows, :, h].double()[..., None, None]).transpose(0, 1).reshape(2, -1, D)[:, :L]
            for k in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = s["q"][starts[b]:starts[b] + n, k].double() @ kv[0].T / math.sqrt(D)
                z += torch.full((n, L), -math.inf, dtype=torch.float64, device=DEV).triu(L - n + 1)
                y[starts[b]:starts[b] + n, k] = torch.softmax(z, 1) @ kv[1]
    return y
