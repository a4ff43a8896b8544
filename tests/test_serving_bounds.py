"""What the long-context tests can see: the bound that outputs are held to
rejects an output that lacks one unit of 32 tokens of its values, and one that
lacks the last token. CPU only."""
import numpy as np
import pytest

from tests import kv8_long as K

SCALE = float(np.float32(1.0 / np.sqrt(128.0)))


@pytest.mark.parametrize("Hkv,L", [(1, 300), (1, 4096), (1, 20000), (8, 20000), (2, 9017)])
@pytest.mark.parametrize("weight_eps,floor", [(2.0 ** -20, 2.0 ** -39), (2.0 ** -11, 2.0 ** -35)])
def test_the_bound_rejects_an_output_without_one_unit(Hkv, L, weight_eps, floor):
    c = K.case(Hkv, Hkv, 32, [1], [L - 1], 7 + L, K.random_codes, K.marked)
    y, _ = K.S.attention(*c, SCALE, weight_eps, None, floor)
    assert K.check_rows(c, y, SCALE, weight_eps, floor) <= 1
    units = -(-L // K.UNIT)
    rng = np.random.default_rng(L)
    for u in {0, 1, units - 2, units - 1, *rng.integers(0, units, 6).tolist()}:
        q, codes, scales, table, lens, start = c
        less = codes.copy()
        less[table[0, u], 1] = 0  # pages of one unit
        short, _ = K.S.attention(q, less, scales, table, lens, start, SCALE, weight_eps, None, floor)
        head = [u // 128 % Hkv]
        assert K.check_rows(c, short, SCALE, weight_eps, floor, heads=head) > 1, u


@pytest.mark.parametrize("L", [33, 300, 4097])
def test_the_bound_rejects_an_output_without_the_last_token(L):
    """(the only one of its unit)"""
    c = K.case(1, 1, 32, [1], [L - 1], L, K.random_codes, K.marked)
    q, codes, scales, table, lens, start = c
    if L % K.UNIT != 1:
        L = L // K.UNIT * K.UNIT + 1
        c = q, codes, scales, table, np.asarray([L], np.int32), start
    y, _ = K.S.attention(q, codes, scales, table, [L - 1], start, SCALE)
    assert K.check_rows(c, y, SCALE, 2.0 ** -11, 2.0 ** -35) > 1
