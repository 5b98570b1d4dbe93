"""Pins for oracle/mxfp4.py and oracle/kv_cache.py: hand-worked codes, scales and pages."""

import numpy as np
import pytest

from exact import bf16_bits_of
from oracle import kv_cache as kvo
from oracle import mxfp4 as m4
from oracle import numerics as nm


def _bits(*vals):
    return np.array([bf16_bits_of(v) for v in vals], np.uint16)


def test_e2m1_ties_and_signs():
    # between two magnitudes the nearer; half way the one with the even code
    v = [0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.0, -0.25, -5.0]
    assert m4.e2m1_encode(np.array(v)).tolist() == [0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 8, 14]
    assert m4.e2m1_decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_block_exponent_borders():
    # 6 fits scale 2^0, the next bf16 does not; the same at 448 and 127; 0 gives the clamp
    assert m4.block_exponent(np.array([6.0, 6.03125, 3.0, 0.0]), 6.0).tolist() == [0, 1, -1, -127]
    assert m4.block_exponent(np.array([448.0, 450.0, 224.0]), 448.0).tolist() == [0, 1, -1]
    assert m4.block_exponent(np.array([127.0, 127.5, 63.5]), 127.0).tolist() == [0, 1, -1]
    assert m4.block_exponent(np.array([2.0 ** -133]), 6.0).tolist() == [-127]


def test_hand_block_and_packing():
    x = np.zeros((1, 1, 32), np.uint16)
    x[0, 0, :4] = _bits(12.0, -1.0, 0.5, 7.0)  # absmax 12: e = 1; 6, -0.5, 0.25 -> 0, 3.5 -> 4
    q, st, byte = m4.group_quant_mxfp4(x)
    assert byte[0, 0, 0] == 128 and q[0, 0, :2].tolist() == [7 | 9 << 4, 0 | 6 << 4]
    assert st.shape == (1, 1, 4) and st[0, 0].tolist() == [128, 0, 0, 0]
    assert m4.values(q, byte)[0, 0, :4].tolist() == [12.0, -1.0, 0.0, 8.0]


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_block_that_is_not_finite(bad):
    x = np.zeros((1, 1, 64), np.uint16)
    x[0, 0, 3] = np.array([bad], np.float32).view(np.uint32)[0] >> 16
    x[0, 0, 40] = _bits(3.0)[0]
    q, st, byte = m4.group_quant_mxfp4(x)
    assert byte[0, 0].tolist() == [255, 126] and not q[0, 0, :16].any()
    assert np.isnan(m4.values(q, byte)[0, 0, :32]).all() and m4.values(q, byte)[0, 0, 40] == 3.0


def test_product_is_the_sum_of_the_values():
    g = np.random.default_rng(1)
    a, ast, ab = m4.group_quant_mxfp4(nm_bits(g.standard_normal((3, 2, 128))))
    w, wst, wb = [], [], []
    for _ in range(2):
        q, s, b = m4.group_quant_mxfp4(nm_bits(g.standard_normal((16, 1, 128))))
        w.append(q[:, 0]), wst.append(s), wb.append(b[:, 0])
    y, _ = m4.product(a, ast, np.stack(w), np.concatenate(wst), a8=False)
    want = np.einsum("mgk,gnk->mgn", m4.values(a, ab), m4.values(np.stack(w), np.stack(wb)))
    assert np.array_equal(y, nm.f64_to_bf16_rn(want))


def nm_bits(x):
    return nm.f64_to_bf16_rn(np.asarray(x, np.float64))


# ---- the cache ---------------------------------------------------------------------------------


def test_spans_of_new_rows():
    assert kvo.spans(5, 20, 16, 4) == [(0, 15, range(0, 1)), (1, 0, range(1, 5))]
    assert kvo.spans(3, 1, 16, 4) == [(0, 0, range(2, 3))]          # two rows before position 0
    assert kvo.spans(40, 40, 16, 2) == [(0, 0, range(0, 16)), (1, 0, range(16, 32))]  # eight behind the table
    assert kvo.spans(0, 7, 16, 4) == []


@pytest.mark.parametrize("dtype", [np.uint8, np.int8])
def test_a_page_whose_scale_grows(dtype):
    codes, scale = np.zeros((16, 2), dtype), np.zeros((1, 1), np.uint8)
    top = kvo.LARGEST[np.dtype(dtype)]
    kvo.put(codes, scale, 0, 0, 0, np.array([[top, 1.0]]))
    assert scale[0, 0] == 127 and kvo.decode(codes[0]).tolist() == [top, 1.0]
    kvo.put(codes, scale, 0, 0, 1, np.array([[4 * top, -8.0]]))
    assert scale[0, 0] == 129                     # a factor of four more
    # int8: 31.75 -> 32, 0.25 -> 0; E4M3: both exact
    assert kvo.decode(codes[:2]).tolist() == [[32.0, 0.0] if dtype == np.int8 else [112.0, 0.25], [top, -2.0]]
    kvo.put(codes, scale, 0, 0, 2, np.array([[1.0, 1.0]]))   # a smaller row keeps the scale
    assert scale[0, 0] == 129
    kvo.put(codes, scale, 0, 0, 0, np.array([[1.0, 1.0]]))   # slot 0: begun anew
    assert scale[0, 0] < 127
    before = codes.copy()
    kvo.put(codes, scale, 0, 0, 3, np.array([[np.nan, 1.0]]))
    assert scale[0, 0] == 255 and not codes[3].any() and np.array_equal(codes[:3], before[:3])


def test_attention_by_hand():
    # one head, D = 64: two keys whose scores differ by log 3, values 0 and 4
    k = np.zeros((1, 1, 16, 64), np.int8)
    v = np.zeros((1, 1, 64, 16), np.int8)
    k[0, 0, 1, 0] = 1
    v[0, 0, :, 1] = 4
    ks = vs = np.full((1, 1), 127, np.uint8)
    q = np.zeros((1, 1, 64), np.uint16)
    q[0, 0, 0] = _bits(1.0)[0]
    o, lse, _, _ = kvo.attention(k, v, ks, vs, q, [0, 1], [2], np.zeros((1, 1), np.int32), np.log(3.0), True)
    assert np.allclose(o, 3.0, rtol=1e-14) and np.allclose(lse, np.log(4.0))
    o, lse, _, _ = kvo.attention(k, v, ks, vs, q, [0, 1], [0], np.zeros((1, 1), np.int32), 1.0, True)
    assert not o.any() and np.isneginf(lse).all()
