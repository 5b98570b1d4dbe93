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


def test_the_largest_magnitudes():
    """From which magnitude on each format rounds up to 2^128, which bf16 reads as infinity."""
    from oracle import mxfp4 as m4

    def back(bits, kind):
        x = np.full((1, 1, 32), bits, np.uint16)
        if kind == "e2m1":
            pairs, _, byte = m4.group_quant_mxfp4(x)
            return m4.values(pairs, byte)[0, 0, 0]
        dtype = np.int8 if kind == "int8" else np.uint8
        c = [np.zeros((1, 1, 16, 64), dtype), np.zeros((1, 1, 64, 16), dtype), np.zeros((1, 1), np.uint8), np.zeros((1, 1), np.uint8)]
        kvo.append(*c, np.full((1, 1, 64), bits, np.uint16), np.full((1, 1, 64), bits, np.uint16), [0, 1], [1], np.zeros((1, 1), int))
        return (kvo.decode(c[0][0, 0, 0]) * m4.scales(c[2][0, 0]))[0]

    for kind, first in (("e2m1", 0x7F60), ("e4m3", 0x7F78), ("int8", 0x7F7F)):
        assert back(first - 1, kind) < 2.0**128 and back(first, kind) == 2.0**128 and back(0x7F7F, kind) == 2.0**128
