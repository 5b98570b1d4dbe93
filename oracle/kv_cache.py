"""Oracle for the paged 8-bit cache: appending rows, and attention over it.

TEST INFRASTRUCTURE ONLY (see the package docstring).

k [pages][H][P][D], v [pages][H][D][P] codes (E4M3 as uint8, or int8), k_scale and v_scale
UE8M0 bytes [pages][H].  Written token by token and row by row from the definitions in wq.h.
"""

from __future__ import annotations

import numpy as np

from .mxfp4 import block_exponent, scales
from .numerics import bf16_to_f32, e4m3_decode, e4m3_encode_rn

LARGEST = {np.dtype(np.uint8): 448.0, np.dtype(np.int8): 127.0}


def decode(codes: np.ndarray) -> np.ndarray:
    return codes.astype(np.float64) if codes.dtype == np.int8 else e4m3_decode(codes)


def encode(v: np.ndarray, dtype) -> np.ndarray:
    return np.rint(v).astype(np.int8) if np.dtype(dtype) == np.int8 else e4m3_encode_rn(v)


def spans(n: int, length: int, P: int, max_pages: int):
    """(page index, first slot, rows) runs of the n newest tokens of a sequence, in order."""
    out, i = [], 0
    while i < n:
        pos = length - n + i
        if pos < 0 or pos >= max_pages * P:
            i += 1
            continue
        run = min(n - i, P - pos % P)
        out.append((pos // P, pos % P, range(i, i + run)))
        i += run
    return out


def append(k, v, k_scale, v_scale, k_new, v_new, offsets, lens, table):
    """k_new, v_new: bf16 bits [T, H, D]; the cache arrays are changed in place."""
    pages, H, P, D = k.shape
    for b in range(len(lens)):
        n = int(offsets[b + 1] - offsets[b])
        for pg, slot, rows in spans(n, int(lens[b]), P, table.shape[1]):
            page = int(table[b, pg])
            if not 0 <= page < pages:
                continue
            for codes, scale, new in ((k[page], k_scale, k_new), (v[page].swapaxes(1, 2), v_scale, v_new)):
                x = bf16_to_f32(new[offsets[b] + rows.start : offsets[b] + rows.stop]).astype(np.float64)
                for h in range(H):
                    put(codes[h], scale, page, h, slot, x[:, h])


def put(codes, scale, page, h, slot, x):
    """x [rows, D] into codes [P, D] (a view) from `slot` on, with the page's scale byte."""
    n = len(x)
    finite = np.isfinite(x).all()
    largest = LARGEST[codes.dtype]
    byte = int(block_exponent(np.abs(x).max(), largest)) + 127 if finite else 255
    if slot > 0:
        old = int(scale[page, h])
        byte = max(byte, old)
        if byte != 255 and byte > old:
            held = codes[:slot]
            nan = (held & 0x7F) == 0x7F if codes.dtype == np.uint8 else np.zeros(held.shape, bool)
            vals = np.ldexp(np.where(nan, 0.0, decode(held)), old - byte)
            codes[:slot] = np.where(nan, held, encode(vals, codes.dtype))
    codes[slot : slot + n] = 0 if byte == 255 else encode(np.ldexp(x, 127 - byte), codes.dtype)
    scale[page, h] = byte


def attention(k, v, k_scale, v_scale, q, offsets, lens, table, scale, causal):
    """q bf16 bits [T, Hq, D] -> (out, lse, mag, smag), f64: out and lse are what the definition
    gives, mag is sum_j softmax_j |v_j| (the scale of the error that rounded weights make), smag
    [T, Hq] the largest scale * sum_d |q_d k_jd| of the keys that a row sees (that of a score's)."""
    pages, H, P, D = k.shape
    T, Hq, _ = q.shape
    qf = bf16_to_f32(q).astype(np.float64)
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, smag = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(lens)):
        n, length = int(offsets[b + 1] - offsets[b]), int(lens[b])
        pos = [p for p in range(max(0, min(length, table.shape[1] * P))) if 0 <= table[b, p // P] < pages]
        pg, sl = table[b, [p // P for p in pos]].astype(int), np.array([p % P for p in pos], int)
        for h in range(Hq):
            c = h // (Hq // H)
            kk = decode(k[pg, c, sl]) * scales(k_scale[pg, c])[:, None]
            vv = decode(v[pg, c, :, sl]) * scales(v_scale[pg, c])[:, None]
            for i in range(n):
                last = length - n + i if causal else length - 1
                see = np.array([p <= last for p in pos], bool)
                if not see.any():
                    continue
                s = scale * (kk[see] @ qf[offsets[b] + i, h])
                m = s.max() if np.isfinite(s).all() else np.nan
                p = np.exp(s - m)
                t = offsets[b] + i
                smag[t, h] = abs(scale) * (np.abs(kk[see]) @ np.abs(qf[t, h])).max()
                lse[t, h] = m + np.log(p.sum())
                out[t, h] = (p / p.sum()) @ vv[see]
                mag[t, h] = (p / p.sum()) @ np.abs(vv[see])
    return out, lse, mag, smag
