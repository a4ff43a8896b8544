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
