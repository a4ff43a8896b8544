"""The append's rotation against its promise (include/w4a8.h): sine and cosine
of p * inv_freq within 2^-23 at every position, for frequencies of any size.

Seen through the page's scale, which is not rounded to fp16: a key whose one
nonzero value is a 1 in its pair is turned into (cos t, sin t) exactly as the
kernel has them (products by 1 and 0), and the scale of its page is fp32(max(
|cos t|, |sin t|) / 127), one rounding (2^-24 relative). So scale * 127 is within
2^-23 + 2^-24 of the exact max(|cos t|, |sin t|) <= 1. t has 48 bits (24 of the
position, 24 of the frequency): exact in 64-bit floating point.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
P, HEADS, B = 128, 64, 48
TOL = 2.0 ** -23 + 2.0 ** -24


@pytest.fixture(autouse=True)
def _no_device_error():
    w4a8.clear_device_error(DEV)
    yield
    assert w4a8.get_device_error(DEV) == 0


def turned(positions, f, interleaved, second, single):
    """max(|cos|, |sin|) as the kernel has it: [positions, pairs]. Head g's key has
    its 1 at pair g (its first or second value)."""
    n = len(f)
    rng = np.random.default_rng(1)
    B = len(positions)
    codes, scales = w4a8.kv8_cache(B, HEADS, P, DEV)
    table = torch.full((B, int(positions.max()) // P + 1), -1, dtype=torch.int32, device=DEV)
    page = rng.permutation(B)
    table[torch.arange(B, device=DEV), torch.from_numpy(positions // P).to(DEV)] = torch.from_numpy(page).int().to(DEV)
    qkv = torch.zeros(B, 3 * HEADS, 128, dtype=torch.float16, device=DEV)
    for g in range(n):
        qkv[:, HEADS + g, 2 * g + second if interleaved else g + second * n] = 1.0
    lens = torch.from_numpy(positions + 1).int().to(DEV)
    start = None if single else torch.arange(B + 1, dtype=torch.int32, device=DEV)
    w4a8.kv8_rope_append(qkv.view(B, -1), HEADS, codes, scales, table, lens, torch.from_numpy(f).to(DEV), q_start=start,
                         interleaved=interleaved)
    return scales.cpu().numpy()[page, 0, :n].astype(np.float64) * 127


def positions(rng):
    p = rng.integers(0, 1 << 24, B)
    p[:6] = 0, 1, 2, (1 << 24) - 1, 131071, 1 << 20
    return p


def check(f, interleaved, second, single, seed):
    p = positions(np.random.default_rng(seed))
    f = np.asarray(f, np.float32)
    t = p[:, None].astype(np.float64) * f.astype(np.float64)
    want = np.maximum(np.abs(np.cos(t)), np.abs(np.sin(t)))
    off = np.abs(turned(p, f, interleaved, second, single) - want)
    assert (off <= TOL).all(), float(off.max() * 2 ** 23)


@pytest.mark.parametrize("interleaved,rotary", [(False, 128), (True, 128), (False, 50), (True, 50)])
@pytest.mark.parametrize("single", [True, False])
def test_angles_of_every_layout(interleaved, rotary, single):
    f = 500000.0 ** (-np.arange(0, rotary, 2) / rotary)
    for second in (0, 1):
        check(f, interleaved, second, single, 10 + rotary + second)


@pytest.mark.parametrize("lo,hi", [(1e-9, 1e-6), (1e-4, 1.0), (1.0, 8.0), (8.0, 1e3), (1e3, 1e6), (1e6, 1e9)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_angles_of_any_frequency(lo, hi, sign):
    """Tiny, ordinary, above one (a base below one) and large frequencies, and turns the other way."""
    rng = np.random.default_rng(20)
    f = sign * np.exp(rng.uniform(np.log(lo), np.log(hi), 64))
    f[0] = sign * hi
    for second in (0, 1):
        check(f, False, second, True, 30 + second)
