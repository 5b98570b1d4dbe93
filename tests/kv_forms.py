"""Sizes that reach each form of the cache's attention, inputs for them, and the definition in
64 bits, a sequence and head at a time (checked against the oracle's row by row in
test_oracle_kv.py)."""

import numpy as np

import synthetic as syn
from oracle import kv_cache as kvo
from oracle import numerics as nm
from oracle.mxfp4 import scales

# new rows and lengths of the sequences, heads, query heads to each, page, pages of a sequence; the
# number that wq_kv_attention_path gives (by heads of 64 and 128, of 256)
FORMS = {
    "items16": dict(ns=[1, 1, 1, 1, 0, 1], lens=[40, 16, 0, 200, 9, 255], H=2, R=4, P=16, width=16, path=(2, 3)),
    "items64": dict(ns=[20, 1, 0, 33, 9], lens=[61, 16, 9, 250, 12], H=2, R=4, P=16, width=16, path=(3, 3)),
    "runs16": dict(ns=[1] * 9, lens=[700, 16, 0, 2040, 33, 1, 512, 64, 1500], H=8, R=4, P=32, width=64, path=(4, 5)),
    "runs64": dict(ns=[20, 1, 0, 13, 40, 9, 1, 30], lens=[700, 16, 9, 1500, 52, 60, 512, 30], H=8, R=4, P=32, width=64, path=(5, 5)),
    "parts16": dict(ns=[1, 1, 1], lens=[9000, 16, 40], H=1, R=4, P=48, width=256, path=(12, 13)),
    "parts64": dict(ns=[20, 9, 3], lens=[3000, 16, 40], H=1, R=4, P=48, width=64, path=(13, 13)),
    "rows": dict(ns=[100, 3, 0, 90, 70], lens=[150, 16, 9, 90, 333], H=8, R=16, P=32, width=12, path=(1, 1)),
}


def form(name, D):
    """Its sizes, offsets and path for heads of D."""
    f = dict(FORMS[name])
    if name == "rows" and D == 256:
        f.update(ns=[60, 3, 0, 40, 30], lens=[90, 16, 9, 40, 333])
    f["path"] = f["path"][D == 256]
    f["offsets"] = np.concatenate(([0], np.cumsum(f["ns"]))).astype(np.int64)
    return f


def cache(g, pages, H, P, D, i8):
    """Any codes but E4M3's NaN, and scales near one."""
    k = g.integers(-127, 128, (pages, H, P, D)).astype(np.int8)
    v = g.integers(-127, 128, (pages, H, D, P)).astype(np.int8)
    if not i8:
        k, v = ((g.integers(0, 0x57, a.shape) | (g.integers(0, 2, a.shape) << 7)).astype(np.uint8) for a in (k, v))
    span = (118, 122) if i8 else (124, 129)
    return k, v, *(g.integers(*span, (pages, H)).astype(np.uint8) for _ in range(2))


def inputs(name, D, i8, seed, extra=2, **kw):
    """(sizes, [k, v, k_scale, v_scale], table, q bits), sizes replaced by kw's."""
    f = dict(form(name, D), **kw)
    f["offsets"] = np.concatenate(([0], np.cumsum(f["ns"]))).astype(np.int64)
    g = syn.rng(80, seed, D, int(i8))
    B = len(f["ns"])
    pages = B * f["width"] + 3
    c = list(cache(g, pages, f["H"], f["P"], D, i8))
    table = g.permutation(pages)[: B * f["width"]].reshape(B, f["width"]).astype(np.int32)
    q = nm.f64_to_bf16_rn(g.standard_normal((int(f["offsets"][-1]) + extra, f["H"] * f["R"], D)))
    return f, c, table, q


def attention(c, q, offsets, lens, table, scale, causal):
    """(out, lse, mag, smag) as kvo.attention has them, and NaN for both out and lse of rows that
    see a page marked NaN or hold one."""
    k, v, ks, vs = c
    pages, H, P, D = k.shape
    T, Hq, _ = q.shape
    R = Hq // H
    qf = nm.bf16_to_f32(q).astype(np.float64)
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, smag = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(lens)):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        n, length = hi - lo, int(lens[b])
        pos = np.arange(max(0, min(length, table.shape[1] * P)))
        pg = table[b, pos // P].astype(np.int64)
        pos, pg = pos[(pg >= 0) & (pg < pages)], pg[(pg >= 0) & (pg < pages)]
        if n == 0 or not len(pos):
            continue
        last = length - n + np.arange(n) if causal else np.full(n, length - 1)
        see = np.repeat(pos[None] <= last[:, None], R, 0)  # [n R, tokens]
        for h in range(H):
            sk, sv = scales(ks[pg, h]), scales(vs[pg, h])
            bad = np.isnan(sk) | np.isnan(sv)
            kk = kvo.decode(k[pg, h, pos % P]) * np.where(bad, 0.0, sk)[:, None]
            vv = kvo.decode(v[pg, h, :, pos % P]) * np.where(bad, 0.0, sv)[:, None]
            x = qf[lo:hi, h * R : h * R + R].reshape(n * R, D)
            lost = (see & bad).any(1) | (np.isnan(x).any(1) & see.any(1))
            x = np.where(np.isnan(x), 0.0, x)
            s = np.where(see, scale * (x @ kk.T), -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
            total = p.sum(1, keepdims=True)
            some = total > 0
            p /= np.where(some, total, 1.0)
            at = np.s_[lo:hi, h * R : h * R + R]
            with np.errstate(divide="ignore"):
                le = np.where(some, m + np.log(total), -np.inf)[:, 0]
            o, w = p @ vv, p @ np.abs(vv)
            smag[at] = np.where(see, abs(scale) * (np.abs(x) @ np.abs(kk).T), 0.0).max(1).reshape(n, R)
            lse[at] = np.where(lost, np.nan, le).reshape(n, R)
            out[at] = np.where(lost[:, None], np.nan, o).reshape(n, R, D)
            mag[at] = w.reshape(n, R, D)
    return out, lse, mag, smag
