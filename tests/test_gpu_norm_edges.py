"""The norm that quantizes at the edges of its formula: rows of nothing
without an eps, quotients midway between two codes, scales beyond fp16. The
rows are chosen so that every value before the codes is exact in fp32 (mean
square and root powers of two), and the expected outputs follow by hand."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
# one width for every thread and vector count
WIDTHS = [512, 2048, 4096, 8192, 16384, 32768, 65536]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.fixture(autouse=True)
def _no_device_error():
    w4a8.clear_device_error(DEV)
    yield
    assert w4a8.get_device_error(DEV) == 0


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_rows_of_zeros_without_an_eps(K, residual):
    """Unused places of a batch are rows of zeros: 0 * rstd is 0 for eps = 0 too."""
    x = np.zeros((3, K), np.float16)
    x[1] = 1.0
    r = dev(-x * np.float16([[0], [0], [1]])) if residual else None
    w = dev(np.full(K, -2.0, np.float16))
    h, codes, s, rowsum = w4a8.rmsnorm_quantize_act(dev(x), w, 0.0, residual=r)
    for row in (0, 2):
        assert not codes[row].any() and float(s[row]) == 0 and int(rowsum[row]) == 0
    assert (codes[1] == -127).all() and float(s[1]) == float(np.float16(2 / 127)) and int(rowsum[1]) == -127 * K


@pytest.mark.parametrize("K", WIDTHS)
def test_quotients_midway_between_two_codes_go_to_the_even_one(K):
    """x of ones, alternating in sign: y is +-w, and w are odd multiples of half
    a scale of 3 / 64. As quantize_act codes the same values."""
    j = np.arange(K)
    w = (3.0 / 128) * (2 * (j % 127) + 1)
    w[5] = 127 * 3.0 / 64
    sign = np.where(j % 3 == 0, -1.0, 1.0)
    x, w16 = sign[None].astype(np.float16), w.astype(np.float16)
    assert (w16 == w).all()
    _, codes, s, rowsum = w4a8.rmsnorm_quantize_act(dev(x), dev(w16), 0.0)
    want = np.rint(sign * w / (3.0 / 64))
    assert float(s[0]) == 3.0 / 64 and (codes[0].cpu().numpy() == want).all() and int(rowsum[0]) == int(want.sum())
    plain, s2, rowsum2 = w4a8.quantize_act(dev((sign * w)[None].astype(np.float16)))
    assert torch.equal(codes, plain) and torch.equal(s, s2) and torch.equal(rowsum, rowsum2)


@pytest.mark.parametrize("K", [16384, 65536])
def test_a_scale_beyond_fp16_is_its_largest_value(K):
    """One value alone in a wide row, under the largest weight: y = sqrt(K) *
    65504 is more than 127 * 65504; sA is 65504 and the code 127, none infinite."""
    x = np.zeros((2, K), np.float16)
    x[0, 3], x[1, K - 1] = 1.0, -2.0
    w = np.full(K, 65504.0, np.float16)
    _, codes, s, rowsum = w4a8.rmsnorm_quantize_act(dev(x), dev(w), 0.0)
    assert (s == 65504).all()
    assert int(codes[0, 3]) == 127 and int(codes[1, K - 1]) == -127 and rowsum.tolist() == [127, -127]
    assert int((codes != 0).sum()) == 2
