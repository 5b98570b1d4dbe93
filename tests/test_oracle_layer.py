"""Pins of the layer's oracle: rows worked by hand, exact arithmetic and identities."""

from fractions import Fraction

import numpy as np
import pytest

import synthetic as syn
from oracle import fp8_group as fg
from oracle import int8_linear as il
from oracle import kv_cache as kvo
from oracle import layer
from oracle import moe
from oracle import numerics as nm


def _bits(a):
    return nm.f64_to_bf16_rn(np.asarray(a, np.float64))


def test_sums_are_the_nearest_bf16_of_the_exact_sum():
    g = syn.rng(90)
    x = _bits(g.standard_normal(4000) * np.exp2(g.integers(-12, 12, 4000)))
    r = _bits(g.standard_normal(4000) * np.exp2(g.integers(-12, 12, 4000)))
    got = nm.bf16_to_f32(layer.add_bf16(x, r))
    for a, b, s in zip(nm.bf16_to_f32(x), nm.bf16_to_f32(r), got):
        exact = Fraction(float(a)) + Fraction(float(b))
        ulp = Fraction(2) ** (max(int(np.floor(np.log2(abs(float(s))))) if s else -126, -126) - 7)
        assert abs(Fraction(float(s)) - exact) <= ulp / 2


def test_sums_that_are_not_finite():
    big = np.array([0x7F7F, 0x7F80, 0x7F80, 0x7FC0, 0xFF7F], np.uint16)
    other = np.array([0x7F7F, 0x3F80, 0xFF80, 0x0000, 0xFF7F], np.uint16)
    assert layer.add_bf16(big, other).tolist() == [0x7F80, 0x7F80, 0x7FC0, 0x7FC0, 0xFF80]


def test_a_row_by_hand():
    # mean square of (3, 1, 3, 1, ...) is 5; eps 4: v = h / 3 * gamma, gamma 1.5 and 3
    h = _bits([[3.0, 1.0] * 16])
    v, other = layer.normed(h, _bits([1.5, 3.0] * 16), 4.0)
    third = np.float32(1) / np.float32(3)
    assert np.array_equal(v[0, :2], [np.float32(3) * third * np.float32(1.5), third * np.float32(3)])
    assert np.array_equal(v, other)
    q, s = layer.rows_int8(v)
    assert q[0, 0] == 127 and q[0, 1] == 85 and s[0] == v[0, 0] / np.float32(127)


@pytest.mark.parametrize("block", [128, 32])
def test_blocks_of_bf16_values_are_the_group_quant(block):
    x = syn.activations((91, block), 5, 640, outlier_frac=0.02, outlier_mul=50.0)
    codes, words = layer.rows_e4m3(nm.bf16_to_f32(x), block)
    want, storage, _ = fg.group_quant_fp8_packed(x[:, None, :], block)
    assert np.array_equal(codes, want[:, 0]) and np.array_equal(words, storage)


def test_what_is_not_finite_stays_in_its_row_or_block():
    x = syn.activations((92,), 4, 256)
    x[1, 3], x[2, 200] = 0x7FC0, 0xFF80
    v, _ = layer.normed(x, _bits(np.ones(256)))
    assert np.isnan(v[1:3]).all() and np.isfinite(v[[0, 3]]).all()
    q, s = layer.rows_int8(v)
    assert np.isnan(s[1:3]).all() and not q[1:3].any() and np.isfinite(s[[0, 3]]).all()
    v[0, 130] = np.inf
    codes, words = layer.rows_e4m3(v, 128)
    byte = fg.unpack_ue8m0(words, 4, 2)[:, 0]
    assert (byte == 255).tolist() == [[False, True], [True, True], [True, True], [False, False]] and not codes[byte.repeat(128, 1) == 255].any()


def test_rows_of_int8_are_the_norms_and_the_quant_of_each():
    x = syn.activations((93,), 3, 128)
    gamma = _bits(1 + 0.1 * syn.rng(94).standard_normal(128))
    v, _ = layer.normed(x, gamma)
    assert np.array_equal(v, moe.rmsnorm_f32(x, gamma))
    assert all(np.array_equal(a, b) for a, b in zip(layer.rows_int8(v), il.quant_int8_per_token(v, is_bf16_bits=False)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_turns(interleaved):
    # a quarter turn exchanges the pair's members exactly; position 0 leaves a row as it is
    x = syn.rng(95).standard_normal((3, 2, 64)).astype(np.float32)
    angles = np.zeros((2, 2, 16), np.float32)
    angles[0, 0], angles[1, 1] = 1.0, 1.0
    y = layer.turned(x, np.array([0, 1, 1]), angles, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[:, :, 32:], x[:, :, 32:])
    one, two = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    assert np.array_equal(y[1:, :, one], -x[1:, :, two]) and np.array_equal(y[1:, :, two], x[1:, :, one])
    # lengths stay, and angles add: turning by p and then q is turning by p + q
    a = np.arange(3)[:, None] * np.exp2(-np.arange(16.0))
    angles = np.stack((np.cos(a), np.sin(a)), 1).astype(np.float32)
    y = layer.turned(layer.turned(x, np.array([1, 1, 1]), angles, interleaved), np.array([1, 0, 1]), angles, interleaved)
    want = layer.turned(x, np.array([2, 1, 2]), angles, interleaved)
    assert np.abs(y - want).max() <= 8 * 2.0**-24 * np.abs(x).max()
    y = layer.turned(x, np.array([-1, 3, 0]), angles, interleaved)
    assert np.isnan(y[:2, :, :32]).all() and np.array_equal(y[:2, :, 32:], x[:2, :, 32:]) and np.isfinite(y[2]).all()


@pytest.mark.parametrize("dtype", [np.int8, np.uint8])
def test_appending_unturned_rows_is_append(dtype):
    g = syn.rng(96)
    H, P, D, ns, lens = 2, 16, 64, [3, 20, 1], [3, 41, 17]
    off = np.concatenate(([0], np.cumsum(ns)))
    table = g.permutation(9).reshape(3, 3)
    angles = np.zeros((41, 2, 32), np.float32)
    angles[:, 0] = 1.0
    kn, vn = (_bits(g.standard_normal((24, H, D))) for _ in range(2))
    caches = []
    for put in range(2):
        c = [np.zeros((9, H, P, D), dtype), np.zeros((9, H, D, P), dtype), np.zeros((9, H), np.uint8), np.zeros((9, H), np.uint8)]
        if put:
            kvo.append(*c, kn, vn, off, lens, table)
        else:
            layer.append_rotated(*c, kn, vn, angles, False, off, lens, table)
        caches.append(c)
    assert all(np.array_equal(a, b) for a, b in zip(*caches))
