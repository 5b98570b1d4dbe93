"""Oracle for the 4-bit microscaled blocks: E2M1 codes, their quantisation, the product.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A block is 32 consecutive elements with one UE8M0 scale.  E2M1 has one sign bit, two
exponent bits (bias 1) and one fraction bit: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 in the
order of their codes; code 8 + c is the negative of code c.  Two codes to a byte, the even
element in the low four bits.
* the exponent is the smallest e with 2^e >= absmax / 6, at least -127;
* the code is the nearest of x * 2^-e, ties to the even code, the sign kept;
* a block with a NaN or an infinity has the scale byte 255 and zero codes, and reads as NaN;
* the product sums the blocks in float64 and rounds once to bf16.
"""

from __future__ import annotations

import numpy as np

from .fp8_group import pack_ue8m0, unpack_ue8m0
from .numerics import bf16_to_f32, e4m3_decode, f64_to_bf16_rn

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def block_exponent(absmax: np.ndarray, largest: float) -> np.ndarray:
    """Smallest e >= -127 with largest * 2^e >= absmax, by exact float64 comparisons."""
    a = np.asarray(absmax, dtype=np.float64)
    e = np.full(a.shape, -127, dtype=np.int64)
    for cand in range(-127, 128):
        e = np.where(np.ldexp(largest, cand) < a, cand + 1, e)
    return e


def e2m1_encode(v: np.ndarray) -> np.ndarray:
    """Values within [-6, 6] -> codes: the nearest magnitude, of two equally near the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    assert np.all(a <= 6.0)
    d = np.abs(a[..., None] - MAGNITUDES)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (pick | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def e2m1_decode(codes: np.ndarray) -> np.ndarray:
    c = np.asarray(codes).astype(np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def pair(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpair(pairs: np.ndarray) -> np.ndarray:
    out = np.empty(pairs.shape[:-1] + (2 * pairs.shape[-1],), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = pairs & 15, pairs >> 4
    return out


def group_quant_mxfp4(x_bits: np.ndarray):
    """bf16 bits [T, G, D] -> (pairs uint8 [T, G, D/2], storage int32 [G, PH, TA], bytes [T, G, D/32])."""
    T, G, D = x_bits.shape
    x = bf16_to_f32(x_bits).astype(np.float64).reshape(T, G, D // BLOCK, BLOCK)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    e = block_exponent(np.abs(x).max(axis=-1, initial=0.0), 6.0)
    codes = e2m1_encode(np.ldexp(x, -e[..., None]))
    codes[bad] = 0
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return pair(codes.reshape(T, G, D)), pack_ue8m0(byte), byte


def scales(byte: np.ndarray) -> np.ndarray:
    """UE8M0 bytes -> float64 powers of two, NaN for 255."""
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))


def values(codes: np.ndarray, byte: np.ndarray, e4m3: bool = False) -> np.ndarray:
    """Codes [.., D/2] pairs or [.., D] E4M3 with scale bytes [.., D/32] -> float64 [.., D]."""
    v = e4m3_decode(codes) if e4m3 else e2m1_decode(unpair(codes))
    return v * np.repeat(scales(byte), BLOCK, axis=-1)


def product(a: np.ndarray, a_storage: np.ndarray, w: np.ndarray, w_storage: np.ndarray, *, a8: bool):
    """a [M, G, K/2] or [M, G, K], w [G, N, K/2], storages [G, K/128, tokens] ->
    (bf16 bits [M, G, N], sum of |terms|)."""
    M, G, _ = a.shape
    N, K = w.shape[1], 2 * w.shape[2]
    av = values(a, unpack_ue8m0(a_storage, M, K // BLOCK), a8)
    out, mag = np.empty((M, G, N)), np.empty((M, G, N))
    for g in range(G):
        wv = values(w[g], unpack_ue8m0(w_storage[g : g + 1], N, K // BLOCK)[:, 0])
        with np.errstate(invalid="ignore"):
            out[:, g], mag[:, g] = av[:, g] @ wv.T, np.abs(av[:, g]) @ np.abs(wv.T)
    return f64_to_bf16_nan(out), mag


def f64_to_bf16_nan(x: np.ndarray) -> np.ndarray:
    """f64 -> bf16 bits, a NaN to 0x7FC0."""
    nan = np.isnan(x)
    return np.where(nan, 0x7FC0, f64_to_bf16_rn(np.where(nan, 0.0, x))).astype(np.uint16)
