"""Workspace sizes of the KV8 attention against the batches that a caller sizes
them for. CPU only."""
import pytest

import w4a8_quantized_gemm_quantize_b200 as w4a8
from w4a8_quantized_gemm_quantize_b200 import build as w4a8_build


@pytest.fixture(scope="module", autouse=True)
def _built():
    w4a8_build.build()


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 8), (8, 1), (64, 8)])
def test_one_more_sequence_does_not_move_a_chunk_to_the_other_kernel(Hq, Hkv):
    """A chunk that is cut along the cache (its parts lie in the workspace) is cut with a sequence of one token
    beside it too: which kernel takes a sequence goes by its own rows."""
    for n in (160 * Hkv // Hq - 1, 41 * Hkv // Hq + 1):
        alone, beside = w4a8.kv8_workspace_bytes(1, n, Hq, Hkv), w4a8.kv8_workspace_bytes(2, n + 1, Hq, Hkv)
        none = w4a8.kv8_workspace_bytes(1, 1, Hkv, Hkv)  # no parts
        assert alone > none and beside > none


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 8), (8, 1), (64, 8), (5, 1), (128, 1), (64, 64), (1024, 1)])
def test_a_workspace_of_the_largest_batch_serves_every_smaller_one(Hq, Hkv):
    size = lambda B, T: w4a8.kv8_workspace_bytes(B, T, Hq, Hkv)  # noqa: E731
    Bs = [1, 2, 3, 4, 8, 9, 16, 18, 19, 32, 64, 300, 65535]
    Ts = [1, 2, 7, 8, 9, 32, 33, 64, 100, 256, 1000, 4096, 100000]
    for B in Bs:
        assert all(size(B, a) <= size(B, b) for a, b in zip(Ts, Ts[1:]))
    for T in Ts:
        assert all(size(a, T) <= size(b, T) for a, b in zip(Bs, Bs[1:]))
    # the parts of a launch are at most one for each of 148 SMs: 256 rows of 128 outputs, a reference and a sum
    assert size(65535, 100000) - w4a8.kv8_decode_workspace_bytes(1, Hq, Hkv) <= 148 * 256 * 130 * 4


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (32, 8), (128, 1)])
def test_a_decode_call_needs_no_parts(Hq, Hkv):
    size = w4a8.kv8_decode_workspace_bytes(1, Hq, Hkv)
    assert size == w4a8.kv8_workspace_bytes(1, 1, 8, 8)  # the partial results alone
    assert w4a8.kv8_decode_workspace_bytes(32, Hq, Hkv) == size == w4a8.kv8_decode_workspace_bytes(65535, Hq, Hkv)
    for bad in ((0, Hq, Hkv), (1, 0, Hkv), (1, Hq, 0), (65536, Hq, Hkv), (1, 3, 2), (1, 1025, 1)):
        assert w4a8.kv8_decode_workspace_bytes(*bad) == 0


def test_counter_bytes_are_the_headers():
    import os
    import re
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a8.h")
    assert int(re.search(r"#define W4A8_KV8_COUNTER_BYTES (\d+)", open(header).read())[1]) == w4a8.KV8_COUNTER_BYTES
