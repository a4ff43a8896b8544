"""Pins of the serving operators' oracle (oracle/serving_oracle.py) on closed
forms, symmetries and hand-worked values. CPU only."""
import numpy as np
import pytest

from oracle import serving_oracle as S

RNG = np.random.default_rng


def test_norm_of_a_constant_row_is_the_weight():
    x = np.full((2, 64), 3.0, np.float16)
    w = np.linspace(-1, 1, 64).astype(np.float16)
    h, y = S.rmsnorm(x, w, 0.0)
    assert np.array_equal(h, x) and np.allclose(y, w.astype(np.float64)[None], rtol=1e-15)


def test_norm_does_not_depend_on_a_power_of_two():
    x = RNG(1).standard_normal((3, 40)).astype(np.float16)
    w = np.ones(40, np.float16)
    a = S.quantize_rows(S.rmsnorm(x, w, 0.0)[1])
    b = S.quantize_rows(S.rmsnorm(x * np.float16(4), w, 0.0)[1])
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_norm_adds_the_residual_with_one_rounding():
    x, r = np.array([[2048.0, 1.0]], np.float16), np.array([[1.0, -1.0]], np.float16)
    h, y = S.rmsnorm(x, np.ones(2, np.float16), 0.0, r)
    assert h[0, 0] == 2048.0 and h[0, 1] == 0.0  # 2049 is halfway: to even
    assert np.allclose(y, [[np.sqrt(2.0), 0.0]])


def test_quantized_rows_of_zeros():
    codes, s = S.quantize_rows(np.zeros((2, 8)))
    assert not codes.any() and not s.any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_positions(interleaved):
    f = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    x = RNG(2).standard_normal((1, 2, 128))
    at = lambda p: S.rotate(x, [p], f, interleaved, 1.0)[0]  # noqa: E731
    assert np.allclose((at(77) ** 2).sum(1), (x[0] ** 2).sum(1))
    assert np.array_equal(at(5)[:, 64:], x[0][:, 64:])  # only 64 of 128 rotated
    dot = lambda a, b: (at(a)[0] * at(b)[1]).sum()  # noqa: E731
    assert np.isclose(dot(3, 10), dot(100003, 100010), rtol=1e-9)


def test_rotation_by_a_quarter_turn():
    x = np.arange(128.0)[None, None]
    y = S.rotate(x, [1], [np.float32(np.pi / 2)], True, 2.0)[0, 0]
    assert np.allclose(y[:2], [-2.0, 0.0], atol=1e-6) and np.array_equal(y[2:], x[0, 0, 2:])
    y = S.rotate(x, [1], np.float32([0, np.pi / 2]), False, 1.0)[0, 0]
    assert np.allclose(y[:4], [0, -3, 2, 1], atol=1e-6)


def test_append_by_hand():
    """Two tokens into a page that holds one, then one into the next page."""
    codes, scales = np.zeros((2, 2, 1, 16, 128), np.int8), np.zeros((2, 2, 1), np.float32)
    codes[1, 0, 0, 13] = 100
    scales[1, 0, 0] = 0.5
    x = np.zeros((3, 3, 128))
    x[0, 1, 0], x[1, 1, 1], x[2, 1, 2] = 127.0, -254.0, 63.5
    want, sc, written = S.append(x, 1, codes, scales, np.array([[1, 0]]), [17], [0, 3])
    assert sc[1, 0, 0] == 2.0 and sc[0, 0, 0] == 0.5 and sc[1, 1, 0] == 0.0
    assert want[1, 0, 0, 13, 0] == 25.0 and want[1, 0, 0, 14, 0] == 63.5 and want[1, 0, 0, 15, 1] == -127.0
    assert want[0, 0, 0, 0, 2] == 127.0 and written[1, 0, 0, 13] == 2 and written[1, 0, 0, 14] == 1
    assert written[0, 0, 0, 0] == 1 and not written[0, 0, 0, 1:].any()


def cache(pages, Hkv, P, seed):
    r = RNG(seed)
    return (r.integers(-127, 128, (pages, 2, Hkv, P, 128)).astype(np.int8),
            (0.01 + 0.02 * r.random((pages, 2, Hkv))).astype(np.float32))


def test_attention_of_one_token_is_its_value():
    codes, scales = cache(3, 2, 16, 3)
    q = RNG(4).standard_normal((1, 4, 128)).astype(np.float16)
    y, _ = S.attention(q, codes, scales, np.array([[2]]), [1], [0, 1], 0.1)
    for h in range(4):
        assert np.allclose(y[0, h], codes[2, 1, h // 2, 0] * scales[2, 1, h // 2].astype(np.float64))


def test_attention_with_zero_queries_is_the_mean_of_what_a_row_sees():
    codes, scales = cache(4, 1, 16, 5)
    table = np.array([[3, 0, 2]])
    y, _ = S.attention(np.zeros((5, 1, 128), np.float16), codes, scales, table, [37], [0, 5], 0.1)
    V = S.gather(codes, scales, table, 0, 37, 0)[1]
    for i in range(5):
        assert np.allclose(y[i, 0], V[:33 + i].mean(0))


def test_attention_does_not_look_behind_the_last_token_or_at_other_pages():
    codes, scales = cache(4, 1, 16, 6)
    q = RNG(7).standard_normal((1, 2, 128)).astype(np.float16)
    table = np.array([[1, 2]])
    a, _ = S.attention(q, codes, scales, table, [20], [0, 1], 0.1)
    codes[2, :, :, 4:], codes[0], scales[3] = 99, 1, np.nan
    b, _ = S.attention(q, codes, scales, table, [20], [0, 1], 0.1)
    assert np.array_equal(a, b)


def test_error_bound_holds_for_fp32_evaluations_and_sees_a_lost_token():
    codes, scales = cache(8, 1, 16, 8)
    table = RNG(9).permutation(8)[None]
    q = RNG(10).standard_normal((1, 1, 128)).astype(np.float16)
    L = 121
    y, E = S.attention(q, codes, scales, table, [L], [0, 1], 0.02)
    K, V = S.gather(codes, scales, table, 0, L, 0)
    f = np.float32
    for seed in range(5):
        o = RNG(seed).permutation(L)
        s = (K[o].astype(f) @ q[0, 0].astype(f)) * f(0.02)
        p = np.exp(s - s.max())
        got = (p @ V[o].astype(f)) / p.sum(dtype=f)
        assert (np.abs(got - y[0, 0]) <= E[0, 0]).all()
    s = 0.02 * (K[1:] @ q[0, 0].astype(np.float64))
    p = np.exp(s - s.max())
    assert (np.abs((p @ V[1:]) / p.sum() - y[0, 0]) > E[0, 0]).any()
