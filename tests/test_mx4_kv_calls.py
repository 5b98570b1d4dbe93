"""The 4-bit and cache calls without a GPU: what the C entries refuse, what the binding
refuses, and the kernels' mapping of workgroups to sequences (restated here) for any offsets.

No kernel runs: every call returns at an argument check.  A zeroed buffer stands in for the
context, of which these checks read nothing but the number of compute units.
"""

import ctypes
import os

import numpy as np
import pytest
import torch

import fp8_dynamic_quant_amd as wq

pytestmark = pytest.mark.skipif(not os.path.exists(wq.LIB_PATH), reason="libwq.so not built")

NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 6


@pytest.fixture()
def ctx():
    return ctypes.create_string_buffer(4096)


P = 0x10000  # a 16-byte aligned address that is never read


@pytest.mark.parametrize("args, want", [
    ((P, 1, 1, 32, P, P), None), ((P, 0, 1, 32, P, P), 0), ((P, -1, 1, 32, P, P), SHAPE), ((P, 1, 0, 32, P, P), SHAPE),
    ((P, 1, 1, 16, P, P), SHAPE), ((P, 1, 65536, 32, P, P), SHAPE), ((P, 1 << 30, 8, 4096, P, P), SHAPE),
    ((None, 1, 1, 32, P, P), NULL), ((P, 1, 1, 32, None, P), NULL), ((P, 1, 1, 32, P, None), NULL),
    ((P + 2, 1, 1, 32, P, P), ALIGN), ((P, 1, 1, 32, P + 8, P), ALIGN), ((P, 1, 1, 32, P, P + 4), ALIGN)])
def test_quant_refusals(ctx, args, want):
    if want is None:
        return
    x, T, G, D, q, s = args
    assert wq.lib().wq_group_quant_mxfp4(ctx, x, T, G, D, q, s, None) == want
    assert wq.lib().wq_group_dequant_mxfp4(ctx, x, q, T, G, D, s, None) == want
    assert wq.lib().wq_group_quant_mxfp4(None, x, T, G, D, q, s, None) == NULL


def _desc(**kw):
    d = wq.MatmulDesc()
    for k, v in dict(dict(payload=4, epilogue=1, M=3, N=32, K=256, batch=1, a=P, lda=128, a_batch_stride=0, a_scale=P,
                          a_scale_tokens=4, b=P, b_batch_stride=0, b_scale=P, y=P, ldy=32, y_batch_stride=0), **kw).items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw, want", [
    (dict(M=0), 0), (dict(N=24), SHAPE), (dict(K=192), SHAPE), (dict(K=131200), SHAPE), (dict(batch=65536), SHAPE),
    (dict(lda=112), SHAPE), (dict(lda=1 << 23), SHAPE), (dict(payload=5), SHAPE), (dict(ldy=16), SHAPE), (dict(a_scale_tokens=3), SHAPE),
    (dict(batch=2, b_batch_stride=16), SHAPE), (dict(a_batch_stride=-16), SHAPE), (dict(y_batch_stride=-8), SHAPE),
    (dict(a=None), NULL), (dict(a_scale=None), NULL), (dict(b=None), NULL), (dict(b_scale=None), NULL),
    (dict(y=None), NULL), (dict(a=P + 8), ALIGN), (dict(lda=136), ALIGN), (dict(ldy=36), ALIGN), (dict(b_scale=P + 4), ALIGN),
    (dict(a_scale=P + 4), ALIGN), (dict(seg_offsets=P), UNSUPPORTED), (dict(acc_out=P), UNSUPPORTED),
    (dict(epilogue=2), UNSUPPORTED), (dict(b_layout=1), UNSUPPORTED), (dict(payload=6), SHAPE)])
def test_product_refusals(ctx, kw, want):
    assert wq.lib().wq_quant_matmul(ctx, ctypes.byref(_desc(**kw)), None) == want


def _cache(**kw):
    d = wq.KvCacheDesc()
    for k, v in dict(dict(code=1, pages=4, heads=2, page_tokens=16, head_dim=64, k=P, v=P, k_scale=P, v_scale=P, table=P,
                          table_stride=4, max_pages=4), **kw).items():
        setattr(d, k, v)
    return d


BAD_CACHES = [
    (dict(code=0), SHAPE), (dict(code=3), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE), (dict(page_tokens=8), SHAPE), (dict(page_tokens=24), SHAPE),
    (dict(page_tokens=272), SHAPE), (dict(head_dim=96), SHAPE), (dict(max_pages=0), SHAPE), (dict(table_stride=3), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k_scale=None), NULL), (dict(v_scale=None), NULL),
    (dict(table=None), NULL), (dict(k=P + 8), ALIGN), (dict(v=P + 8), ALIGN)]


def _append(ctx, cache, k=P, ldk=128, v=P, ldv=128, T=5, B=2, off=P, lens=P):
    return wq.lib().wq_kv_append(ctx, ctypes.byref(cache), k, ldk, v, ldv, T, B, off, lens, None)


def _attend(ctx, cache, q=P, ldq=512, T=5, heads=8, B=2, off=P, lens=P, scale=1.0, causal=1, out=P, ldo=512, ws=None, n=0):
    return wq.lib().wq_kv_attention(ctx, ctypes.byref(cache), q, ldq, T, heads, B, off, lens, scale, causal, out, ldo,
                                    None, ws, n, None)


@pytest.mark.parametrize("kw, want", BAD_CACHES)
def test_cache_refusals(ctx, kw, want):
    assert _append(ctx, _cache(**kw)) == want
    assert _attend(ctx, _cache(**kw)) == want


@pytest.mark.parametrize("kw, want", [
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(ldk=120), SHAPE), (dict(ldv=120), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(off=None), NULL), (dict(lens=None), NULL), (dict(ldk=132), ALIGN),
    (dict(k=P + 2), ALIGN), (dict(v=P + 2), ALIGN), (dict(ldv=132), ALIGN)])
def test_append_refusals(ctx, kw, want):
    assert _append(ctx, _cache(), **kw) == want
    assert _append(None, _cache(), **kw) == NULL


@pytest.mark.parametrize("kw, want", [
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), SHAPE), (dict(heads=1), SHAPE), (dict(heads=3), SHAPE), (dict(ldq=504), SHAPE),
    (dict(ldo=504), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(q=P + 2), ALIGN), (dict(out=P + 8), ALIGN), (dict(ldq=516), ALIGN), (dict(ws=P + 4), ALIGN)])
def test_attention_refusals(ctx, kw, want):
    assert _attend(ctx, _cache(), **kw) == want
    assert _attend(None, _cache(), **kw) == NULL


def test_attention_workspace(ctx):
    L = wq.lib()
    cus = 256
    # num_cu is the context's second int
    ctypes.memmove(ctypes.addressof(ctx) + 4, ctypes.byref(ctypes.c_int(cus)), 4)
    one = _cache(max_pages=8192, table_stride=8192)
    need = L.wq_kv_attention_workspace_bytes(ctx, ctypes.byref(one), 1, 8, 1)
    assert 0 < need <= 64 << 20
    for T, B, pages in ((1, 1, 1 << 20), (7, 3, 1 << 20), (64, 64, 4096), (513, 1, 4096), (1, 300, 1 << 16)):
        for heads in (1, 2, 8):
            for D in (64, 128, 256):
                big = _cache(max_pages=pages, table_stride=pages, heads=heads, head_dim=D)
                assert 0 <= L.wq_kv_attention_workspace_bytes(ctx, ctypes.byref(big), T, heads * 16, B) <= 64 << 20
    assert _attend(ctx, one, T=1, B=1, ws=P, n=need - 1) == WORKSPACE
    assert L.wq_kv_attention_workspace_bytes(ctx, ctypes.byref(one), 0, 8, 1) == 0
    assert L.wq_kv_attention_workspace_bytes(ctx, ctypes.byref(one), 1, 3, 1) == -SHAPE
    assert L.wq_kv_attention_workspace_bytes(None, ctypes.byref(one), 1, 8, 1) == -NULL


def test_attention_refuses_rows_beyond_31_bits(ctx):
    one = _cache(heads=1)
    need = lambda T, heads: wq.lib().wq_kv_attention_workspace_bytes(ctx, ctypes.byref(one), T, heads, 1)  # noqa: E731
    assert need(1 << 27, 16) == -SHAPE and need((1 << 27) - 1, 16) >= 0
    assert _attend(ctx, one, T=1 << 30, heads=2, ldq=1 << 20, ldo=1 << 20) == SHAPE


def test_binding_refusals():
    x = torch.zeros((3, 1, 64), dtype=torch.bfloat16)
    for bad in (x.float(), x[0], x.transpose(0, 2), torch.zeros((3, 1, 48), dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            wq.wq_group_quant_mxfp4(bad)
    q, st = torch.zeros((3, 1, 32), dtype=torch.uint8), torch.zeros((1, 1, 4), dtype=torch.int32)
    for a, b in ((q.int(), st), (q, st.float()), (q, st[:, :, :3]), (q[:, :, :24], st)):
        with pytest.raises(ValueError):
            wq.wq_group_dequant_mxfp4(a, b)
    a, sa = torch.zeros((3, 1, 64), dtype=torch.uint8), torch.zeros((1, 1, 4), dtype=torch.int32)
    w, sw = torch.zeros((1, 16, 64), dtype=torch.uint8), torch.zeros((1, 1, 16), dtype=torch.int32)
    for args, kw in (((a[:, :, :32], sa, w, sw), {}), ((a, sa[:, :, :3], w, sw), {}), ((a, sa, w, sa), {}),
                     ((a, sa, w.int(), sw), {}), ((a, sa, w, sw), dict(acc_out=sa)), ((a, sa, w, sw), dict(epilogue=2))):
        with pytest.raises(ValueError):
            wq.wq_quant_matmul(*args, fp8_groups=1, mx4=True, **kw)
    with pytest.raises(ValueError):
        wq.wq_quant_matmul(a, sa, w, sw, mx4=True)

    c = wq.kv_cache(4, 2, 16, 64, device="cpu")
    row = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    off, lens, tab = torch.tensor([0, 3]), torch.tensor([3], dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    for bad in (dict(k=row.float()), dict(k=row[:, :1]), dict(k=row[:2]), dict(offsets=off.int()), dict(offsets=off[:1]),
                dict(lens=lens.long()), dict(table=tab.long()), dict(table=tab[:, None]),
                dict(cache=c._replace(v=c.k)), dict(cache=c._replace(v=c.v.view(torch.int8))),
                dict(cache=c._replace(k_scale=c.k_scale.int())), dict(cache=c._replace(k=c.k.transpose(2, 3)))):
        with pytest.raises(ValueError):
            wq.wq_kv_append(**dict(dict(cache=c, k=row, v=row, offsets=off, lens=lens, table=tab), **bad))
    for bad in (dict(q=row.float()), dict(q=row[0]), dict(q=row[:, :, :32]), dict(out=row[:2]), dict(out=row.float()),
                dict(lse=torch.zeros(3, 2, dtype=torch.float64)), dict(lens=lens.long())):
        with pytest.raises(ValueError):
            wq.wq_kv_attention(**dict(dict(cache=c, q=row, offsets=off, lens=lens, table=tab), **bad))


# ---- the mapping of slots to sequences, restated ------------------------------------------------


def find_slot(offsets, T, item, mul, div, per):
    """Last sequence whose first slot is not behind `item`, as the kernels search it."""
    off = lambda b: min(max(int(offsets[b]), 0), T)  # noqa: E731
    lo, hi = 0, len(offsets) - 2
    while lo < hi:
        mid = (lo + hi + 1) >> 1
        if off(mid) * mul // div + per * mid <= item:
            lo = mid
        else:
            hi = mid - 1
    j = item - (off(lo) * mul // div + per * lo)
    return lo, off(lo), (off(lo + 1) - off(lo)) if j >= 0 else 0, max(j, 0)


def append_slots(T, B, page):
    return T // page + 2 * B


@pytest.mark.parametrize("seed", range(60))
def test_every_new_row_has_one_slot(seed):
    from oracle import kv_cache as kvo

    g = np.random.default_rng(seed)
    B, page = int(g.integers(1, 9)), int(g.choice([16, 32, 48, 256]))
    n = g.integers(0, 70, B) * (g.random(B) < 0.8)
    offsets = np.concatenate(([0], np.cumsum(n)))
    T = int(offsets[-1] + g.integers(0, 5))
    lens, max_pages = g.integers(-3, 200, B), int(g.integers(1, 6))
    got = []
    for item in range(append_slots(T, B, page)):
        b, row0, rows, j = find_slot(offsets, T, item, 1, page, 2)
        if rows <= 0:
            continue
        start = int(lens[b]) - rows
        pg = max(start, 0) // page + j
        lo, hi = max(start, pg * page), min(int(lens[b]), (pg + 1) * page)
        if lo >= hi or pg >= max_pages:
            continue
        got.append((b, pg, lo - pg * page, range(lo - start, hi - start)))
        assert 0 <= row0 + lo - start and row0 + hi - start <= T
    want = [(b, *s) for b in range(B) for s in kvo.spans(int(n[b]), int(lens[b]), page, max_pages)]
    assert sorted(got, key=str) == sorted(want, key=str)


def find_slot_256(offsets, T, item, div, per):
    """The same by rounds of 256 sequences, as append's workgroups search it."""
    off = lambda b: min(max(int(offsets[b]), 0), T)  # noqa: E731
    lo, span = 0, len(offsets) - 1
    while True:
        step = (span + 255) // 256
        votes = sum(off(lo + i) // div + per * (lo + i) <= item for i in range(0, 256 * step, step) if i < span)
        at = max(votes - 1, 0)
        if step == 1:
            base = off(lo + at) // div + per * (lo + at)
            return lo + at, off(lo + at), 0 if item < base else off(lo + at + 1) - off(lo + at), max(item - base, 0)
        lo, span = lo + at * step, min(step, span - at * step)


@pytest.mark.parametrize("seed", range(40))
def test_slots_of_append_by_rows_or_by_pages(seed):
    from oracle import kv_cache as kvo

    g = np.random.default_rng(300 + seed)
    B, page = int(g.choice([1, 5, 255, 256, 257, 600])), int(g.choice([16, 48]))
    n = g.integers(0, int(g.choice([2, 3, 90])), B) * (g.random(B) < 0.7)
    offsets = np.concatenate(([0], np.cumsum(n)))
    T = int(offsets[-1] + g.integers(0, 5))
    lens, max_pages = n + g.integers(-3, 90, B), int(g.integers(1, 9))
    by_rows = T <= append_slots(T, B, page)
    div, per = (1, 0) if by_rows else (page, 2)
    got = []
    for item in range(T if by_rows else append_slots(T, B, page)):
        b, row0, rows, j = find_slot_256(offsets, T, item, div, per)
        if rows <= 0:
            continue
        start = int(lens[b]) - rows
        pg = max(start, 0) // page + j
        lo, hi = max(start, pg * page), min(int(lens[b]), (pg + 1) * page)
        if lo >= hi or pg >= max_pages:
            continue
        assert 0 <= row0 + lo - start and row0 + hi - start <= T
        got.append((b, pg, lo - pg * page, range(lo - start, hi - start)))
    want = [(b, *s) for b in range(B) for s in kvo.spans(int(n[b]), int(lens[b]), page, max_pages)]
    assert sorted(got, key=str) == sorted(want, key=str)


@pytest.mark.parametrize("seed", range(20))
def test_append_of_offsets_that_hold_anything_stays_in_bounds(seed):
    g = np.random.default_rng(400 + seed)
    B, T, page = int(g.choice([1, 7, 300])), int(g.integers(1, 100)), 16
    offsets, lens = g.integers(-50, 150, B + 1), g.integers(-20, 200, B)
    for div, per in ((1, 0), (page, 2)):
        for item in range(T if per == 0 else append_slots(T, B, page)):
            b, row0, rows, j = find_slot_256(offsets, T, item, div, per)
            assert 0 <= b < B
            if rows <= 0:
                continue
            start = int(lens[b]) - rows
            pg = max(start, 0) // page + j
            lo, hi = max(start, pg * page), min(int(lens[b]), (pg + 1) * page)
            if lo < hi:
                assert 0 <= row0 + lo - start and row0 + hi - start <= T


@pytest.mark.parametrize("seed", range(60))
def test_every_query_row_has_one_tile(seed):
    g = np.random.default_rng(100 + seed)
    B, R, tile = int(g.integers(1, 9)), int(g.choice([1, 2, 3, 5, 16, 40])), int(g.choice([16, 64, 128]))
    n = g.integers(0, 50, B) * (g.random(B) < 0.7)
    offsets = np.concatenate(([0], np.cumsum(n)))
    T = int(offsets[-1] + g.integers(0, 5))
    seen = []
    for item in range(T * R // tile + B):
        b, row0, rows, j = find_slot(offsets, T, item, R, tile, 1)
        for r in range(j * tile, min((j + 1) * tile, rows * R)):
            seen.append((row0 + r // R, r % R))
    assert sorted(seen) == [(t, r) for t in range(int(offsets[-1])) for r in range(R)]


@pytest.mark.parametrize("seed", range(40))
def test_offsets_that_hold_anything_stay_in_bounds(seed):
    g = np.random.default_rng(200 + seed)
    B, T, R, tile = int(g.integers(1, 9)), int(g.integers(1, 100)), int(g.integers(1, 9)), 16
    offsets = g.integers(-50, 150, B + 1)
    for item in range(T * R // tile + B):
        b, row0, rows, j = find_slot(offsets, T, item, R, tile, 1)
        assert 0 <= b < B
        for r in range(j * tile, min((j + 1) * tile, rows * R)):
            assert r >= 0 and 0 <= row0 + r // R < T


# ---- equal runs of attention's work, restated -----------------------------------------------------


def attention_runs(ns, lens, heads, R, krows, most, least, fixed, cut, capacity):
    """What each workgroup computes, and which parts each join adds: {item: [(step, n, slot)]},
    {item: [slot]}."""
    steps = [max(-(-min(max(x, 0), capacity) // 64), 1) for x in lens]
    units_of = lambda s: s + fixed if cut else 1  # noqa: E731
    pre = np.concatenate(([0], np.cumsum([-(-n * R // krows) * units_of(s) for n, s in zip(ns, steps)]))).tolist()
    units = pre[-1] * heads
    per = max(-(-units // most), least)
    runs = -(-units // per)

    def item_of(u):
        b = max(i for i in range(len(ns)) if pre[i] * heads <= u)
        n = units_of(steps[b])
        item = (u - pre[b] * heads) // n
        i0 = pre[b] * heads + item * n
        tiles = (pre[b + 1] - pre[b]) // n
        return (b, item // tiles, item % tiles), steps[b], (max(u - i0 - fixed, 0) if cut else 0), i0

    done, joins = {}, {}
    for w in range(runs):
        u, end, part = w * per, min((w + 1) * per, units), 0
        while u < end:
            it, s, step, i0 = item_of(u)
            n = (min(max(end - i0 - fixed, 0), s) if cut else s) - step
            if n <= 0:
                break
            done.setdefault(it, []).append((step, n, 2 * w + min(part, 1)))
            u, part = i0 + units_of(s), part + 1
        if cut and w > 0:
            it, s, step, i0 = item_of(w * per)
            before = (w - 1) * per
            if step > 0 and before <= i0 + fixed:
                last = (i0 + fixed + s - 1) // per
                joins[it] = [2 * (w - 1) + (before < i0)] + [2 * (w - 1 + p) for p in range(1, last - w + 2)]
    assert runs <= most
    return done, joins


@pytest.mark.parametrize("seed", range(80))
def test_runs_cover_every_item_once(seed):
    g = np.random.default_rng(300 + seed)
    B, heads, R, krows = int(g.integers(1, 10)), int(g.integers(1, 6)), int(g.choice([1, 4, 5, 16])), int(g.choice([16, 64]))
    ns = (g.integers(0, 20, B) * (g.random(B) < 0.8)).tolist()
    if sum(ns) == 0:
        ns[0] = 1
    lens, cut = g.integers(-3, 4000, B).tolist(), bool(g.random() < 0.8)
    tiles = sum(-(-n * R // krows) for n in ns)
    most = int(g.integers(1, 200)) if cut else tiles * heads
    done, joins = attention_runs(ns, lens, heads, R, krows, most, int(g.choice([4, 8])) if cut else 1, int(g.choice([0, 4, 8])), cut,
                                 int(g.choice([64, 1000, 10000])))
    assert len(done) == tiles * heads
    for it, parts in done.items():
        at = 0
        for step, n, _ in parts:
            assert step == at
            at += n
        assert len(parts) == 1 or joins.pop(it) == [slot for _, _, slot in parts]
    assert not joins
