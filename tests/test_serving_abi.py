"""Refusals of the serving operators, on the host and before any CUDA call;
frequencies for long contexts against their formulas. CPU only."""
import ctypes
import math

import numpy as np
import pytest

import w4a8_quantized_gemm_quantize_b200 as w4a8
from w4a8_quantized_gemm_quantize_b200 import build as w4a8_build

torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced: validation fails first
ODD = 0x10001


@pytest.fixture(scope="module")
def L():
    w4a8_build.build()
    return w4a8.lib()


def test_rmsnorm_refusals(L):
    def call(X=FAKE, r=FAKE, w=FAKE, eps=1e-5, M=4, K=128, H=FAKE, A8=FAKE, sA=FAKE, rs=FAKE):
        return L.w4a8_rmsnorm_quantize_act(X, r, w, eps, M, K, H, A8, sA, rs, None)

    assert call(K=7) == 2 and call(K=0) == 2 and call(K=65544) == 2
    assert call(M=-1) == 1 and call(X=None) == 1 and call(w=None) == 1
    assert call(H=None) == 1 and call(r=None) == 1      # H exactly with a residual
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(X=ODD) == 3 and call(w=ODD) == 3 and call(r=ODD) == 3 and call(H=ODD) == 3 and call(A8=ODD) == 3
    assert call(M=0, X=None) == 0


def desc(**kw):
    d = dict(codes=FAKE, scales=FAKE, block_table=FAKE, num_pages=8, max_blocks=4, Hkv=2, page=64, D=128, reserved=0)
    d.update(kw)
    return w4a8.Kv8CacheDesc(*(d[f] for f, _ in w4a8.Kv8CacheDesc._fields_))


BAD_CACHES = [(dict(D=64), 2), (dict(page=48), 2), (dict(page=8), 2), (dict(Hkv=0), 2), (dict(Hkv=3), 2),
              (dict(Hkv=-1), 1), (dict(num_pages=0), 2), (dict(num_pages=-1), 1), (dict(max_blocks=0), 2),
              (dict(max_blocks=(1 << 24) // 64 + 1), 2), (dict(num_pages=1 << 24), 2), (dict(reserved=1), 1),
              (dict(num_pages=1 << 62), 2), (dict(max_blocks=1 << 62), 2), (dict(num_pages=(1 << 31) // 256), 2),
              (dict(codes=None), 1), (dict(scales=None), 1), (dict(block_table=None), 1), (dict(codes=FAKE + 64), 3),
              (dict(scales=ODD), 3), (dict(block_table=ODD), 3)]


def append(L, c, lens=FAKE, start=FAKE, B=2, T=5, Hq=4, f=FAKE, rd=128, inter=0, ms=1.0, qkv=FAKE, q=FAKE):
    return L.w4a8_kv8_rope_append(qkv, c, lens, start, B, T, Hq, f, rd, inter, ms, q, None)


def decode(L, c, q=FAKE, lens=FAKE, B=2, Hq=4, out=FAKE, ws=FAKE, n=1 << 30):
    return L.w4a8_kv8_attention_decode(q, c, lens, B, Hq, 1.0, out, ws, n, None)


def prefill(L, c, q=FAKE, lens=FAKE, start=FAKE, B=2, T=5, Hq=4, out=FAKE, ws=FAKE, n=1 << 30):
    return L.w4a8_kv8_attention_prefill(q, c, lens, start, B, T, Hq, 1.0, out, ws, n, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(L, kw, status):
    c = desc(**kw)
    assert append(L, c) == status and decode(L, c) == status and prefill(L, c) == status


def test_kv8_refusals(L):
    c = desc()
    assert append(L, None) == 1 and decode(L, None) == 1 and prefill(L, None) == 1
    for f in (append, decode, prefill):
        assert f(L, c, B=-1) == 1 and f(L, c, B=65536) == 2 and f(L, c, Hq=3) == 2 and f(L, c, Hq=1026) == 2
        assert f(L, c, lens=None) == 1 and f(L, c, lens=ODD) == 3 and f(L, c, q=None) == 1 and f(L, c, q=ODD) == 3
        assert f(L, c, B=0) == 0
    assert append(L, c, rd=130) == 2 and append(L, c, rd=63) == 2 and append(L, c, rd=-2) == 2
    assert append(L, c, inter=2) == 1 and append(L, c, f=None) == 1 and append(L, c, f=ODD) == 3
    assert append(L, c, qkv=None) == 1 and append(L, c, qkv=ODD) == 3
    assert append(L, c, start=None) == 1               # one row per sequence: T must be B
    assert append(L, c, start=ODD) == 3 and append(L, c, T=-1) == 1 and append(L, c, T=0) == 0
    assert append(L, c, T=1 << 30) == 2
    assert prefill(L, c, start=None) == 1 and prefill(L, c, start=ODD) == 3 and prefill(L, c, T=0) == 0
    for f in (decode, prefill):
        assert f(L, c, out=None) == 1 and f(L, c, out=ODD) == 3
        assert f(L, c, ws=None) == 4 and f(L, c, n=16) == 4 and f(L, c, ws=FAKE + 16) == 3
    ws = L.w4a8_kv8_attention_workspace_bytes
    assert ws(0, 1, 4, 2) == 0 and ws(1, 0, 4, 2) == 0 and ws(1, 1, 3, 2) == 0 and ws(4, 4, 32, 8) > 0
    assert prefill(L, c, n=ws(2, 5, 4, 2) - 1) == 4


def test_binding_refuses_cpu_tensors_and_bad_arguments():
    h = torch.zeros((2, 128), dtype=torch.float16)
    with pytest.raises(w4a8.W4A8Error):
        w4a8.rmsnorm_quantize_act(h, h[0], 1e-5)
    codes, scales = w4a8.kv8_cache(2, 1, 16)
    i32 = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(w4a8.W4A8Error):
        w4a8.kv8_attention_decode(h.view(2, 1, 128), codes, scales, i32, i32[0], 1.0)
    with pytest.raises(w4a8.W4A8Error):
        w4a8.kv8_attention_prefill(h.view(2, 1, 128), codes, scales, i32, i32[0], None, 1.0)
    with pytest.raises(w4a8.W4A8Error):
        w4a8.kv8_rope_append(h, 1, codes, scales, i32, i32[0], torch.zeros(64))
    for bad in ((0, 1, 16), (1, 0, 16), (1, 1, 48)):
        with pytest.raises(w4a8.W4A8Error):
            w4a8.kv8_cache(*bad)


def test_rope_frequencies():
    f, ms = w4a8.rope_frequencies(128, 500000.0)
    j = np.arange(64)
    plain = 500000.0 ** (-j / 64)
    assert ms == 1.0 and f.dtype == torch.float32 and np.allclose(f.numpy(), plain, rtol=1e-7)
    f, ms = w4a8.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert ms == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32) / 4, rtol=1e-7)
    f, ms = w4a8.rope_frequencies(128, 500000.0, "bands", 8.0, 8192)
    turns = 8192 * plain / (2 * math.pi)
    got = f.numpy().astype(np.float64)
    assert ms == 1.0 and np.allclose(got[turns > 4], plain[turns > 4], rtol=1e-7)
    assert np.allclose(got[turns < 1], plain[turns < 1] / 8, rtol=1e-7)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((got[mid] > plain[mid] / 8) & (got[mid] < plain[mid])).all()
    f, ms = w4a8.rope_frequencies(128, 10000.0, "ramp", 16.0, 4096)
    got = f.numpy().astype(np.float64)
    plain = 10000.0 ** (-j / 64)
    assert math.isclose(ms, 0.1 * math.log(16) + 1) and np.allclose(got[0], plain[0]) and np.allclose(got[-1], plain[-1] / 16)
    assert (np.diff(got / plain) <= 1e-7).all()
    for bad in ((130,), (63,), (128, -1.0), (128, 1e4, "none", 0.5), (128, 1e4, "nothing")):
        with pytest.raises(w4a8.W4A8Error):
            w4a8.rope_frequencies(*bad)
