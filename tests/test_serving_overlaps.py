"""Buffers that overlap where a kernel would read what it has overwritten are
refused on the host. CPU only: the buffers are addresses, never touched."""
import pytest

import w4a8_quantized_gemm_quantize_b200 as w4a8
from w4a8_quantized_gemm_quantize_b200 import build as w4a8_build

BASE, FAR = 1 << 20, 1 << 40
INVALID, WORKSPACE = 1, 4


@pytest.fixture(scope="module")
def L():
    w4a8_build.build()
    return w4a8.lib()


def cache(Hkv=2):
    d = dict(codes=FAR, scales=FAR, block_table=FAR, num_pages=8, max_blocks=4, Hkv=Hkv, page=64, D=128, reserved=0)
    return w4a8.Kv8CacheDesc(*(d[f] for f, _ in w4a8.Kv8CacheDesc._fields_))


@pytest.mark.parametrize("at", [-16, 16, 2 * 4 * 128 - 16, 16 - 2 * 4 * 128])
@pytest.mark.parametrize("over", ["X", "residual"])
def test_norm_refuses_an_h_across_its_input(L, at, over):
    other = 2 * BASE
    X, r = (BASE, other) if over == "X" else (other, BASE)
    assert L.w4a8_rmsnorm_quantize_act(X, r, FAR, 1e-5, 4, 128, BASE + at, FAR, FAR, FAR, None) == INVALID


@pytest.mark.parametrize("at", [0, 16, 5 * 8 * 256 - 16, 16 - 5 * 4 * 256])
def test_append_refuses_queries_over_its_rows(L, at):
    """4 + 2 x 2 heads, 5 rows: 10240 bytes of qkv, 5120 of q_out."""
    for start, T, B in ((FAR, 5, 2), (None, 5, 5)):
        assert L.w4a8_kv8_rope_append(BASE, cache(), FAR, start, B, T, 4, FAR, 128, 0, 1.0, BASE + at, None) == INVALID


@pytest.mark.parametrize("at", [16, -16, 5 * 4 * 256 - 16, 16 - 5 * 4 * 256])
def test_attention_refuses_an_output_across_the_queries(L, at):
    ws = 1 << 30
    assert L.w4a8_kv8_attention_prefill(BASE, cache(), FAR, FAR, 2, 5, 4, 1.0, BASE + at, FAR, ws, None) == INVALID
    assert L.w4a8_kv8_attention_decode(BASE, cache(), FAR, 5, 4, 1.0, BASE + at, FAR, ws, None) == INVALID


def test_neighbours_and_the_same_buffer_are_no_overlap(L):
    """Refused for their workspace alone, which is looked at later."""
    n = 5 * 4 * 256
    for out in (BASE, BASE + n, BASE - n):
        assert L.w4a8_kv8_attention_prefill(BASE, cache(), FAR, FAR, 2, 5, 4, 1.0, out, FAR, 16, None) == WORKSPACE
        assert L.w4a8_kv8_attention_decode(BASE, cache(), FAR, 5, 4, 1.0, out, FAR, 16, None) == WORKSPACE
