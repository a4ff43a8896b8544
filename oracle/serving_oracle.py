"""CPU oracle for the serving operators — TEST INFRASTRUCTURE ONLY.

The norm that quantizes, the rotary append into a paged 8-bit KV cache and
attention over it, in 64 bits and in plain loops over sequences, pages and
heads. Only the tests import this module; it shares no code with the
product.

Definitions (stated in include/w4a8.h):

* norm: h = fp16(x + r); y = h / sqrt(mean h^2 + eps) * w; s = fp16(max |y| /
  127); codes = clamp(rint(y / s), -127, 127).
* cache: int8 codes [pages, 2, Hkv, P, 128], one scale per (page, K | V,
  head); token p of sequence b at place p % P of page table[b, p // P].
* append: the page's scale grows to max(s, max |new| / 127), s = 0 where the
  page's first place is new; codes that were there are carried over.
* attention: row i of n new tokens of a sequence of length L sees its first
  L - n + i + 1 tokens.
"""
from __future__ import annotations

import numpy as np

D = 128
U = 2.0 ** -23  # covers rounded and truncated fp32 operations


def rmsnorm(x, w, eps, r=None):
    """(h fp16, y float64): the residual stream and the norm's exact values."""
    h = np.asarray(x, np.float16)
    if r is not None:
        h = (h.astype(np.float64) + np.asarray(r, np.float16).astype(np.float64)).astype(np.float16)
    v = h.astype(np.float64)
    y = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * np.asarray(w, np.float16).astype(np.float64)
    return h, y


def quantize_rows(y):
    """(codes int8, s fp16) of rows y float64."""
    s = (np.abs(y).max(axis=1) / 127).astype(np.float16)
    sf = s.astype(np.float64)[:, None]
    codes = np.where(sf > 0, np.clip(np.rint(y / np.where(sf > 0, sf, 1)), -127, 127), 0)
    return codes.astype(np.int8), s


def rotate(x, positions, inv_freq, interleaved, ms):
    """x [T, heads, 128] float64 rotated at positions [T]."""
    x = np.array(x, np.float64)
    n = len(inv_freq)
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float32).astype(np.float64)
    c, s = np.cos(t)[:, None] * ms, np.sin(t)[:, None] * ms
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = a * s + b * c
    return x


def spans(q_start, seq_lens):
    """(first row, new tokens, position of the first) of each sequence."""
    return [(int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(L) - int(q_start[b + 1] - q_start[b]))
            for b, L in enumerate(seq_lens)]


def append(x, Hq, codes, scales, table, seq_lens, q_start):
    """The cache after appending the (rotated) rows x [T, Hq + 2 Hkv, 128]:
    (values before rounding to codes in units of the scale, i.e. x / s' or c *
    (s / s'), float64 like codes; scales float64; written: places that hold
    new tokens, 2: places carried over)."""
    Hkv, P = codes.shape[2], codes.shape[3]
    want, sc = codes.astype(np.float64), scales.astype(np.float64)
    written = np.zeros(codes.shape[:4], np.int8)
    for b, (first, n, pos0) in enumerate(spans(q_start, seq_lens)):
        if n <= 0:
            continue
        for p in range(pos0 // P, (pos0 + n - 1) // P + 1):
            lo, hi = max(pos0, p * P), min(pos0 + n, (p + 1) * P)
            page = int(table[b, p])
            for kv in range(2):
                for g in range(Hkv):
                    v = x[first + lo - pos0:first + hi - pos0, Hq + kv * Hkv + g]
                    old = sc[page, kv, g] if lo > p * P else 0.0
                    new = max(old, np.abs(v).max() / 127)
                    a, e = lo - p * P, hi - p * P
                    if new > old:
                        want[page, kv, g, :a] *= old / new
                        written[page, kv, g, :a] = 2
                    want[page, kv, g, a:e] = v / new if new > 0 else 0.0
                    written[page, kv, g, a:e] = 1
                    sc[page, kv, g] = new
    return want, sc, written


def gather(codes, scales, table, b, L, g):
    """K and V float64 [2, L, 128] of one sequence and kv head."""
    P = codes.shape[3]
    rows = np.asarray(table[b, :-(-L // P)], np.int64)
    v = codes[rows][:, :, g].astype(np.float64) * scales[rows][:, :, g].astype(np.float64)[..., None, None]
    return v.transpose(1, 0, 2, 3).reshape(2, -1, D)[:, :L]


def attention(q, codes, scales, table, seq_lens, q_start, scale, weight_eps=0.0, heads=None, weight_floor=0.0):
    """(y, E) float64 [T, Hq, 128]: the exact outputs and a bound on what an
    fp32 evaluation in any order and split may be off by, with the softmax
    weights of the numerator rounded to `weight_eps` relative, or, where that
    is more, by `weight_floor` of the row's largest weight. Rows of no sequence
    are NaN. u = 2^-23:

    * a score: products exact (11-bit by 8-bit significands), their 128-term sum
      gamma_128 sum |q c|, three rounded factors: delta_j = scale * sK * gamma_131
      * sum |q c|.
    * a weight exp(s_j - m) sV_j: the argument off by 2 delta + 8 u (|s_j - m| +
      |log2 sV_j|) (subtractions, changes of the exponent's base, rescales), the
      exponentials and products by 16 u: relative error R_j. The same error in
      numerator and denominator moves y by at most sum p R |V - y| / sum p (1 -
      R); the numerator's own rounding by weight_eps * sum p |V| / sum p.
    * the sums over L tokens with at most L / 16 rescales, partial results
      merged, the division: gamma_{2 L + 64} (sum p |V| / sum p + |y|)."""
    q = np.asarray(q, np.float16).astype(np.float64)
    T, Hq, _ = q.shape
    Hkv = codes.shape[2]
    y, E = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    for b, (first, n, pos0) in enumerate(spans(q_start, seq_lens)):
        L = int(seq_lens[b])
        for h in (range(Hq) if heads is None else heads):
            if n <= 0:
                continue
            if L == 0:
                y[first:first + n, h] = 0
                continue
            K, V = gather(codes, scales, table, b, L, h // (Hq // Hkv))
            sv = np.repeat(scales[np.asarray(table[b, :-(-L // codes.shape[3])], np.int64), 1, h // (Hq // Hkv)],
                           codes.shape[3])[:L].astype(np.float64)
            rows = np.asarray(table[b, :-(-L // codes.shape[3])], np.int64)
            C = np.abs(codes[rows, 1, h // (Hq // Hkv)].reshape(-1, D)[:L].astype(np.float64))
            for i in range(n):
                m = pos0 + i + 1
                s = scale * (K[:m] @ q[first + i, h])
                p = np.exp(s - s.max())
                o = (p @ V[:m]) / p.sum()
                y[first + i, h] = o
                d = abs(scale) * 131 * U * (np.abs(K[:m]) @ np.abs(q[first + i, h]))
                lg = np.abs(np.log2(np.maximum(sv[:m], 1e-30)))
                R = np.expm1(2 * d.max() + 8 * U * (np.abs(s - s.max()) + lg) + 16 * U)
                a = (p @ np.abs(V[:m])) / p.sum()
                e = (p * R) @ np.abs(V[:m] - o) / (p * (1 - np.minimum(R, 0.5))).sum() + weight_eps * a
                if weight_floor:
                    e = e + weight_floor * (p * sv[:m]).max() * C[:m].sum(axis=0) / p.sum()
                E[first + i, h] = 1.1 * (e + (2 * m + 64) * U * (a + np.abs(o)))
    return y, E
