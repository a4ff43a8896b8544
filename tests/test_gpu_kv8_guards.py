"""KV8 attention writes its outputs and its workspace and nothing else: guard
regions before and after both, rows of no sequence, workspaces of the size that
the size functions say."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests import test_gpu_kv8 as T  # noqa: E402
from tests.test_gpu_kv8 import _no_device_error  # noqa: E402,F401

DEV, SCALE = T.DEV, T.SCALE
GUARD = 4096


def guarded(nbytes, fill):
    """A buffer of nbytes between guards, and what checks the guards."""
    b = torch.full((nbytes + 2 * GUARD,), fill, dtype=torch.uint8, device=DEV)

    def intact():
        return bool((b[:GUARD] == fill).all()) and bool((b[GUARD + nbytes:] == fill).all())
    return b[GUARD:GUARD + nbytes], intact


def run_guarded(c, decode):
    q, codes, scales, table, lens, start = (T.dev(a) for a in c)
    rows, Hq, Hkv, B = q.shape[0], q.shape[1], codes.shape[2], len(lens)
    out, out_ok = guarded(q.numel() * 2, 0x5A)
    out = out.view(torch.float16).view(q.shape).fill_(7.0)
    need = w4a8.kv8_decode_workspace_bytes(B, Hq, Hkv) if decode else w4a8.kv8_workspace_bytes(B, rows, Hq, Hkv)
    ws, ws_ok = guarded(need, 0x7F)
    ws[:w4a8.KV8_COUNTER_BYTES] = 0
    for _ in range(2):
        if decode:
            w4a8.kv8_attention_decode(q, codes, scales, table, lens, SCALE, out=out, workspace=ws)
        else:
            w4a8.kv8_attention_prefill(q, codes, scales, table, lens, start, SCALE, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert out_ok() and ws_ok() and not ws[:w4a8.KV8_COUNTER_BYTES].any()
    with pytest.raises(w4a8.W4A8Error):
        if decode:
            w4a8.kv8_attention_decode(q, codes, scales, table, lens, SCALE, out=out, workspace=ws[:need - 1])
        else:
            w4a8.kv8_attention_prefill(q, codes, scales, table, lens, start, SCALE, out=out, workspace=ws[:1024])
    return T.host(out)


@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 1, [70] * 32), (4, 4, [1, 0, 5000]), (32, 8, [1]), (36, 3, [333, 2100, 17])])
def test_decode_writes_only_its_outputs(Hq, Hkv, lens):
    """With the decode call's own size, which holds no parts of the other kernel."""
    c = list(T.case(Hq, Hkv, 16, [1] * len(lens), [max(n - 1, 0) for n in lens], 70 + Hq))
    c[4] = T.i32(lens)
    T.check_attention(c, run_guarded(c, True), 2.0 ** -20, heads=(0, Hq - 1))


@pytest.mark.parametrize("Hq,Hkv,new,old", [(4, 1, [5], [90]), (4, 1, [300, 2, 70], [900, 60, 0]), (32, 8, [257, 130], [0, 40]),
                                            (3, 1, [100], [5000])])
def test_prefill_writes_only_its_outputs(Hq, Hkv, new, old):
    """A few rows, pieces cut along the cache, whole ones, an odd group; padding rows behind."""
    c = T.case(Hq, Hkv, 32, new, old, 80 + Hq + new[0], pad_rows=5)
    T.check_attention(c, run_guarded(c, False), 2.0 ** -11, heads=(0, Hq - 1))


def test_one_workspace_for_the_largest_batch():
    """Sized for the longest chunk and the most sequences, used for shorter and fewer, and for single tokens."""
    ws = torch.zeros(w4a8.kv8_workspace_bytes(4, 1200, 4, 1), dtype=torch.uint8, device=DEV)
    for new, old in (([1000, 100], [10, 3]), ([64], [3000]), ([9], [500]), ([1, 1, 1, 1], [5, 70, 900, 31])):
        c = T.case(4, 1, 32, new, old, 90 + len(new))
        T.check_attention(c, T.attend(c, False, ws), 2.0 ** -11, heads=(0, 3))
        if max(new) == 1:
            T.check_attention(c, T.attend(c, True, ws), 2.0 ** -20)
