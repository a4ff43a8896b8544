"""The norm that quantizes (w4a8_rmsnorm_quantize_act) against the oracle in
64 bits.

Tolerances, derived: the fp32 sum of squares adds at most 64 terms per thread
and 5 + 32 partial sums (relative error under 101 * 2^-24), halved by the
root; the division, the sum with eps, the root, the reciprocal and the two
products by rstd and w add at most 7 roundings more: y is within REL = 2^-18
of its exact value, relatively. So the scale is the fp16 rounding of a value
within REL of max |y| / 127, and with the scale taken as given a code is
within 1/2 + 127 * (REL + 2^-24) of y / s (before the clamp).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_quantized_gemm_quantize_b200 as w4a8
from w4a8_quantized_gemm_quantize_b200 import inputs as I
from oracle import serving_oracle as S
from oracle import w4a8_oracle as O
from tests._util import max_ulp_fp16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
REL = 2.0 ** -18
EPS = 1e-5


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.fixture(autouse=True)
def _no_device_error():
    w4a8.clear_device_error(DEV)
    yield
    assert w4a8.get_device_error(DEV) == 0


def check(x, w, r, eps, got):
    h, y = S.rmsnorm(x, w, eps, r)
    H, A8, sA, rs = (None if t is None else t.cpu().numpy() for t in got)
    if r is None:
        assert H is None
    else:
        assert np.array_equal(H.view(np.uint16) & 0x7FFF, h.view(np.uint16) & 0x7FFF) and np.array_equal(H, h)
    top = np.abs(y).max(axis=1) / 127
    lo, hi = (top * (1 - 2 * REL)).astype(np.float16), (top * (1 + 2 * REL)).astype(np.float16)
    assert ((sA >= lo) & (sA <= hi)).all()
    sf = sA.astype(np.float64)[:, None]
    q = np.where(sf > 0, y / np.where(sf > 0, sf, 1), 0)
    assert (np.abs(A8) <= 127).all()
    assert (np.abs(np.clip(q, -127, 127) - A8) <= 0.5 + 127 * (REL + 2.0 ** -24) * np.maximum(1, np.abs(q) / 127)).all()
    assert np.array_equal(rs, A8.sum(axis=1, dtype=np.int64))


def draw(M, K, seed, residual=True):
    x = I.activations(M, K, seed)
    r = I.activations(M, K, seed + 1) if residual else None
    w = (1 + 0.1 * np.random.default_rng(seed + 2).standard_normal(K)).astype(np.float16)
    return x, w, r


# every thread count and vector count, their edges, and one row to many
@pytest.mark.parametrize("M,K", [(1, 8), (3, 64), (2, 1024), (5, 1032), (7, 2048), (3, 2056), (33, 4096), (2, 4104),
                                 (3, 8192), (2, 8200), (3, 14336), (2, 16384), (2, 16392), (1, 32768), (2, 32776),
                                 (1, 65536), (300, 1000), (1, 4096), (65, 4096)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_matches_the_oracle(M, K, residual):
    x, w, r = draw(M, K, I.seed_of("norm", M, K), residual)
    check(x, w, r, EPS, w4a8.rmsnorm_quantize_act(dev(x), dev(w), EPS, residual=None if r is None else dev(r)))


def test_norm_special_rows():
    """Zero rows (with and without eps: 0 / 0 is not met, y = 0 * rstd), rows
    of the smallest and of large values, one spike, opposite residuals."""
    K = 512
    x = np.zeros((6, K), np.float16)
    x[1] = np.float16(6e-8)
    x[2] = 200.0
    x[3, 77] = 60000.0
    x[4] = np.linspace(-1, 1, K)
    x[5] = 1.0
    r = np.zeros_like(x)
    r[4] = -x[4]
    w = np.linspace(-2, 2, K).astype(np.float16)
    got = w4a8.rmsnorm_quantize_act(dev(x), dev(w), 1e-6, residual=dev(r))
    check(x, w, r, 1e-6, got)
    assert not got[1][0].any() and float(got[2][0]) == 0 and not got[1][4].any()
    zero_w = w4a8.rmsnorm_quantize_act(dev(x), torch.zeros(K, dtype=torch.float16, device=DEV), 1e-6)
    assert not zero_w[1].any() and not zero_w[2].any() and not zero_w[3].any()


@pytest.mark.parametrize("alias", ["x", "residual"])
def test_norm_in_place_and_twice(alias):
    """H may be X or the residual; a second call on H alone gives the same codes."""
    x, w, r = draw(40, 4096, 17)
    X, R, W = dev(x), dev(r), dev(w)
    ref = w4a8.rmsnorm_quantize_act(X, W, EPS, residual=R)
    H = {"x": X, "residual": R}[alias]
    out = (H, *(torch.empty_like(t) for t in ref[1:]))
    got = w4a8.rmsnorm_quantize_act(X, W, EPS, residual=R, out=out)
    again = w4a8.rmsnorm_quantize_act(H, W, EPS)
    assert got[0].data_ptr() == H.data_ptr()
    for a, b, c in zip(ref[1:], got[1:], again[1:]):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert torch.equal(ref[0], H)


def test_norm_writes_only_its_outputs():
    M, K = 5, 1000
    x, w, r = draw(M, K, 23)
    pad = 64
    bufs = [torch.full((M * K + 2 * pad,), v, dtype=t, device=DEV) for v, t in ((7.0, torch.float16), (7, torch.int8))]
    rows = [torch.full((M + 2 * pad,), 7, dtype=t, device=DEV) for t in (torch.float16, torch.int32)]
    out = (bufs[0][pad:-pad].view(M, K), bufs[1][pad:-pad].view(M, K), rows[0][pad:-pad], rows[1][pad:-pad])
    check(x, w, r, EPS, w4a8.rmsnorm_quantize_act(dev(x), dev(w), EPS, residual=dev(r), out=out))
    for b in bufs + rows:
        assert (b[:pad] == 7).all() and (b[-pad:] == 7).all()


def test_norm_feeds_the_gemm():
    """norm -> GEMM: the GEMM of the codes that the norm wrote, against the
    oracle's GEMM of the same codes (1 ulp, as for the quantizer's)."""
    M, N, K = 16, 256, 512
    x, w, r = draw(M, K, 31)
    codes = I.uniform_codes(N, K, 32)
    blob = w4a8.pack_weights(*(dev(c) for c in codes))
    H, A8, sA, rs = w4a8.rmsnorm_quantize_act(dev(x), dev(w), EPS, residual=dev(r))
    Y = w4a8.gemm(A8, sA, rs, blob, N, K)
    want = O.epilogue(O.gemm_acc(A8.cpu().numpy(), O.dequant_weights(*codes[:3])), sA.cpu().numpy(), codes[3])
    assert max_ulp_fp16(Y.cpu().numpy(), want) <= 1


def test_norm_on_another_stream_and_in_a_graph():
    x, w, r = draw(9, 4096, 41)
    X, W, R = dev(x), dev(w), dev(r)
    ref = w4a8.rmsnorm_quantize_act(X, W, EPS, residual=R)
    out = tuple(torch.empty_like(t) for t in ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w4a8.rmsnorm_quantize_act(X, W, EPS, residual=R, out=out)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4a8.rmsnorm_quantize_act(X, W, EPS, residual=R, out=out)
    x2, _, r2 = draw(9, 4096, 43)
    X.copy_(dev(x2))
    R.copy_(dev(r2))
    g.replay()
    torch.cuda.synchronize()
    check(x2, w, r2, EPS, out)


def test_norm_refuses_mismatched_tensors():
    x, w, r = (dev(a) for a in draw(4, 256, 51))
    bad = [dict(X=x.float()), dict(X=x[:, ::2]), dict(weight=w[:128]), dict(weight=w.float()), dict(residual=r[:2]),
           dict(residual=r.cpu()), dict(out=(x, x, w, w)),
           dict(out=(None, x.to(torch.int8), x[:, 0].contiguous(), x[:, 0].int()))]
    for kw in bad:
        a = dict(X=x, weight=w, eps=EPS, residual=r)
        a.update(kw)
        with pytest.raises(w4a8.W4A8Error):
            w4a8.rmsnorm_quantize_act(**a)
    with pytest.raises(w4a8.W4A8Error):
        w4a8.rmsnorm_quantize_act(x[:, :100].contiguous(), w[:100].contiguous(), EPS)  # K % 8
