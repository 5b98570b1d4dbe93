"""The definition of the cache's attention a sequence and head at a time (kv_forms) against the
oracle's row by row."""

import numpy as np
import pytest

import kv_forms as kf
from oracle import kv_cache as kvo


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("name", ["items16", "items64"])
def test_the_two_definitions_agree(name, i8, causal):
    f, c, table, q = kf.inputs(name, 64, i8, 1)
    table[0, 1], table[3, 0] = -1, 1 << 30
    args = (q, f["offsets"], f["lens"], table, -0.125, causal)
    for got, want in zip(kf.attention(c, *args), kvo.attention(*c, *args)):
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        ok = ~np.isneginf(want)
        assert np.allclose(got[ok], want[ok], rtol=1e-12, atol=1e-13)


def test_rows_that_see_a_nan():
    f, c, table, q = kf.inputs("items64", 64, True, 2)
    c[2][table[1, 0], 1] = 255   # keys of the one page of a sequence
    c[3][table[3, 15], 0] = 255  # values of the last page of another, that its last rows see
    q[0, 5, 3] = 0x7FC0
    out, lse, _, _ = kf.attention(c, q, f["offsets"], f["lens"], table, 0.125, True)
    want = np.zeros(lse.shape, bool)
    want[0, 5] = want[20, 4:] = True
    want[21 + np.arange(33)[250 - 33 + np.arange(33) >= 240], :4] = True
    assert np.array_equal(np.isnan(lse), want) and np.array_equal(np.isnan(out).all(-1), want)
    assert np.array_equal(np.isnan(out).any(-1), want)
