"""Oracle for what stands between a layer's products: the residual's addition with the norm and
the 8-bit rows, and rows appended to the paged cache with their keys turned by position.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Written from the definitions in wq.h:
* h = bf16(x + residual); v = (h * inv) * gamma as in moe (the same reading of the sum of squares:
  a row whose f32 mean square another float64 order could round otherwise is flagged, and both
  are accepted); rows in int8 with a scale each, or E4M3 blocks of 128 or 32 with UE8M0 bytes;
* a pair (a, b) becomes (a c - b s, b c + a s) in f32, every product and sum rounded; keys go to
  their codes unrounded, queries are rounded to bf16.
"""

from __future__ import annotations

import numpy as np

from . import kv_cache as kvo
from . import moe
from .fp8_group import pack_ue8m0
from .int8_linear import quant_int8_per_token
from .mxfp4 import block_exponent
from .numerics import bf16_to_f32, e4m3_encode_rn, f64_to_bf16_rn


def add_bf16(x_bits: np.ndarray, r_bits: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        s = bf16_to_f32(x_bits).astype(np.float64) + bf16_to_f32(r_bits).astype(np.float64)
    out = f64_to_bf16_rn(np.where(np.isfinite(s), s, 0.0))
    out = np.where(np.isposinf(s), 0x7F80, np.where(np.isneginf(s), 0xFF80, out))
    return np.where(np.isnan(s), 0x7FC0, out).astype(np.uint16)


def normed(h_bits: np.ndarray, gamma_bits: np.ndarray, eps=1e-6):
    """(v, v_other) f32 [M, K]; rows that hold what is not finite are NaN."""
    bad = ~np.isfinite(bf16_to_f32(h_bits)).all(1)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        v, other, _ = moe.rmsnorm_f32(np.where(bad[:, None], 0, h_bits).astype(np.uint16), gamma_bits, np.float32(eps), alternates=True)
    v[bad] = other[bad] = np.nan
    return v, other


def rows_int8(v: np.ndarray):
    """(codes int8, scales f32): NaN and zeros for rows that hold what is not finite."""
    bad = ~np.isfinite(v).all(1)
    q, s = quant_int8_per_token(np.where(bad[:, None], np.float32(0), v), is_bf16_bits=False)
    s[bad] = np.nan
    return q, s


def rows_e4m3(v: np.ndarray, block: int):
    """(codes uint8 [M, K], words int32 [1, PH, TA])."""
    M, K = v.shape
    b = v.astype(np.float64).reshape(M, K // block, block)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = block_exponent(np.abs(b).max(-1), 448.0)
    codes = e4m3_encode_rn(np.ldexp(b, -e[..., None])).reshape(M, K)
    codes = np.where(np.repeat(bad, block, 1), 0, codes).astype(np.uint8)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes, pack_ue8m0(byte[:, None, :])


def turned(x: np.ndarray, positions: np.ndarray, angles: np.ndarray, interleaved: bool) -> np.ndarray:
    """f32 rows [T, heads, D] at their positions, angles f32 [positions, 2, rot / 2]; NaN where a
    position has no angle."""
    x = x.astype(np.float32).copy()
    half = angles.shape[2]
    fine = (positions >= 0) & (positions < len(angles))
    cs = angles[np.where(fine, positions, 0)]
    cs = np.where(fine[:, None, None], cs, np.float32(np.nan))
    c, s = cs[:, None, 0], cs[:, None, 1]
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., one].copy(), x[..., two].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., one] = a * c - b * s  # f32 throughout: each operation rounds
        x[..., two] = b * c + a * s
    return x


def positions_of(offsets, lens) -> np.ndarray:
    """Position of every row that a sequence has."""
    return np.concatenate([int(lens[b]) - int(offsets[b + 1] - offsets[b]) + np.arange(int(offsets[b + 1] - offsets[b]))
                           for b in range(len(lens))]).astype(np.int64)


def append_rotated(k, v, k_scale, v_scale, k_new, v_new, angles, interleaved, offsets, lens, table):
    """kv_cache.append with the keys turned; bf16 bits in, the cache arrays changed in place."""
    pages, H, P, D = k.shape
    n = int(offsets[-1])
    keys = turned(bf16_to_f32(k_new[:n]), positions_of(offsets, lens), angles, interleaved).astype(np.float64)
    values = bf16_to_f32(v_new[:n]).astype(np.float64)
    for b in range(len(lens)):
        for pg, slot, rows in kvo.spans(int(offsets[b + 1] - offsets[b]), int(lens[b]), P, table.shape[1]):
            page = int(table[b, pg])
            if not 0 <= page < pages:
                continue
            at = slice(int(offsets[b]) + rows.start, int(offsets[b]) + rows.stop)
            for codes, scale, x in ((k[page], k_scale, keys[at]), (v[page].swapaxes(1, 2), v_scale, values[at])):
                for h in range(H):
                    kvo.put(codes[h], scale, page, h, slot, x[:, h])
