"""The bounds-checked debug build on the KV8 append and attention: every
instantiation, ragged edges, cut pieces, results joined across CTAs. The
results must match the oracle with the device error word clear; lengths, starts
and pages that do not fit are reported as such, not as an access out of bounds."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests import test_gpu_kv8 as T  # noqa: E402
from tests.test_gpu_debug_build import debug_lib  # noqa: E402,F401


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("rotary,interleaved", [(128, False), (50, False), (64, True)])
def test_debug_append(debug_lib, P, rotary, interleaved):  # noqa: F811
    T.check_append(6, 2, P, [1] * 5, [0, P - 1, P, 1000, 3], rotary, interleaved, 1.0, P)
    T.check_append(6, 2, P, [70, 1, 0, 129], [0, P - 1, 9, 200], rotary, interleaved, 1.0, P + 1, pad_rows=3)


def test_debug_append_many_rows(debug_lib):  # noqa: F811
    T.check_append(2, 1, 64, [700, 801], [0, 30], 128, False, 1.0, 302)


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 1), (36, 3)])
@pytest.mark.parametrize("P", [16, 128])
def test_debug_decode(debug_lib, Hq, Hkv, P):  # noqa: F811
    c = T.case(Hq, Hkv, P, [1] * 4, [0, 31, 700, 9000], 10 * Hq + P)
    T.check_attention(c, T.attend(c, True), 2.0 ** -20, heads=(0, Hq - 1))


@pytest.mark.parametrize("Hq,Hkv,new,old", [(4, 1, [300, 0, 19], [5000, 40, 700]), (32, 8, [1, 300, 8, 130], [500, 70, 0, 31]),
                                            (6, 2, [3, 9, 0, 1], [100, 5, 7, 0]), (3, 1, [1000], [500])])
def test_debug_prefill(debug_lib, Hq, Hkv, new, old):  # noqa: F811
    c = T.case(Hq, Hkv, 32, new, old, 600 + Hq, pad_rows=3)
    T.check_attention(c, T.attend(c, False), 2.0 ** -11, heads=(0, Hq - 1))


def test_debug_bad_lengths_starts_and_pages_stay_in_bounds(debug_lib):  # noqa: F811
    c = list(T.case(4, 2, 16, [90, 9, 70], [20, 30, 40], 31))
    c[3], c[4], c[5] = c[3].copy(), c[4].copy(), c[5].copy()
    c[4][0], c[3][1, 0], c[5][2] = 1 << 20, -5, 60
    g = [T.dev(a) for a in c]
    w4a8.kv8_attention_prefill(*g, T.SCALE)
    assert w4a8.get_device_error(T.DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(T.DEV)
    w4a8.kv8_attention_decode(g[0][:3].contiguous(), *g[1:5], T.SCALE)
    assert w4a8.get_device_error(T.DEV) == w4a8.DEVERR_KV_RANGE
    w4a8.clear_device_error(T.DEV)
