"""What the serving kernels' sources must hold where no run can show its lack:
the order of tensor-memory accesses behind a wait. CPU only."""
import os
import re

import w4a8_quantized_gemm_quantize_b200 as w4a8

CSRC = os.path.join(os.path.dirname(w4a8.__file__), "csrc")


def lines(name):
    """The source's lines without comments, with their brace depth at the start."""
    depth, out = 0, []
    for text in open(os.path.join(CSRC, name)):
        text = re.sub(r"//.*", "", text).strip()
        out.append((depth - text.startswith("}"), text))
        depth += text.count("{") - text.count("}")
    return out


# barriers that tcgen05.commit arrives on, or that stand for tensor memory
# another thread has written or read
TENSOR_BARS = r"k(SFull|SRead|PFull|PFree)\b"
TENSOR_OPS = r"\b(tmem_ld_\w+|tmem_st_\w+|mma_f16_\w+)\("
FENCE = r"\btc_fence_after\(\)"


def test_prefill_fences_between_each_wait_and_tensor_memory():
    """A wait on a barrier of the tensor-core pipeline is followed by the tcgen05
    fence before the next access to tensor memory, on every path: the fence is
    no deeper in conditions than one level inside the wait's own statement."""
    code = lines("kv8_prefill.cuh")
    body = next(i for i, (_, s) in enumerate(code) if "kv8_prefill_kernel(" in s)
    waits = [i for i in range(body, len(code)) if re.search(r"\bwait\w*\(" + TENSOR_BARS, code[i][1])]
    assert len(waits) >= 5
    for i in waits:
        fence = next((k for k in range(i, len(code)) if re.search(FENCE, code[k][1])), None)
        access = next((k for k in range(i + 1, len(code)) if re.search(TENSOR_OPS, code[k][1])), len(code))
        assert fence is not None and fence < access, code[i][1]
        opens = code[i][1].endswith("{")  # the wait opens the block that the fence stands in
        assert code[fence][0] <= code[i][0] + opens, (code[i][1], "the fence is conditional")
