"""GPU parity of the paged 8-bit cache: appended codes and scales bit for bit, attention within
what its roundings allow."""

import numpy as np
import pytest
import torch

import synthetic as syn
from gpu_util import DEV, assert_same, bf16_dev, dev, host, host_bf16_bits, poison
from oracle import kv_cache as kvo
from oracle import numerics as nm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


def _cache(g, pages, H, P, D, i8):
    """Any codes but E4M3's NaN, and scales near one."""
    k = g.integers(-127, 128, (pages, H, P, D)).astype(np.int8)
    v = g.integers(-127, 128, (pages, H, D, P)).astype(np.int8)
    if not i8:
        # magnitudes around 2^-4 .. 2^3, either sign, with zeros and subnormals among them
        k, v = ((g.integers(0, 0x57, a.shape) | (g.integers(0, 2, a.shape) << 7)).astype(np.uint8) for a in (k, v))
    span = (118, 122) if i8 else (124, 129)
    return k, v, *(g.integers(*span, (pages, H)).astype(np.uint8) for _ in range(2))


def _table(g, B, max_pages, pages):
    return g.permutation(pages)[: B * max_pages].reshape(B, max_pages).astype(np.int32)


def _devs(*arrays):
    return [dev(a) for a in arrays]


def _rows(g, T, H, D, loud=0.0):
    return nm.f64_to_bf16_rn(g.standard_normal((T, H, D)) * np.exp2(loud * g.standard_normal((T, 1, 1))))


def _append_check(seed, i8, P, D, H, ns, lens, max_pages, *, loud=2.0, spoil=None, pad=0, extra=0):
    g = syn.rng(50, seed)
    B = len(ns)
    pages = B * max_pages + 2
    k, v, ks, vs = _cache(g, pages, H, P, D, i8)
    table = _table(g, B, max_pages, pages)
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    T = int(off[-1]) + extra
    kn, vn = _rows(g, T, H, D, loud), _rows(g, T, H, D, loud)
    if spoil:
        spoil(table, kn, vn)
    c = wq.KvCache(*_devs(k, v, ks, vs))
    wide = torch.full((T, H * D + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, : H * D] = bf16_dev(kn).view(T, H * D)
    kd = wide[:, : H * D].unflatten(1, (H, D))
    args = (c, kd, bf16_dev(vn), dev(off), dev(np.array(lens, np.int32)), dev(table))
    print(f"append i8={i8} P={P} D={D} H={H} n={ns} lens={lens}", flush=True)
    wq.wq_kv_append(*args)
    torch.cuda.synchronize()
    kvo.append(k, v, ks, vs, kn, vn, off, lens, table)
    for twice in (False, True):
        for name, got, want in zip(("k", "v", "k_scale", "v_scale"), c, (k, v, ks, vs)):
            assert_same(name + (" again" if twice else ""), host(got), want)
        if not twice:  # the same call again writes the same bytes
            wq.wq_kv_append(*args)
            torch.cuda.synchronize()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("P", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_lengths(i8, P, D):
    # one row at a page's start, inside, at its end; runs over a border; whole pages; nothing
    _append_check(P + D, i8, P, D, 2, [1, 1, 1, 0, 3, P, P + 5, 2 * P + 1], [1, 2, P, 9, P + 1, P, 2 * P + 2, 2 * P + 1], 3)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("H, D", [(1, 64), (3, 128), (8, 128), (5, 256)])
def test_append_heads_in_wider_rows(i8, H, D):
    _append_check(H, i8, 32, D, H, [4, 1, 40], [30, 33, 41], 2, pad=24, extra=3)


@pytest.mark.parametrize("i8", [False, True])
def test_append_of_rows_much_larger_and_much_smaller(i8):
    for seed, loud in ((1, 12.0), (2, 0.0)):
        _append_check(seed, i8, 64, 128, 2, [1] * 12 + [5], list(range(7, 19)) + [64], 2, loud=loud)


@pytest.mark.parametrize("i8", [False, True])
def test_append_beyond_the_table_and_before_the_first_token(i8):
    _append_check(3, i8, 16, 64, 2, [20, 7, 5, 4], [37, 3, 0, -2], 2)


@pytest.mark.parametrize("i8", [False, True])
def test_append_to_pages_that_are_none(i8):
    def spoil(table, kn, vn):
        table[0, 0], table[1, 1], table[2, 0] = -1, 1 << 30, len(table) * 2 + 2

    _append_check(4, i8, 16, 64, 2, [20, 20, 3, 2], [20, 25, 3, 2], 2, spoil=spoil)


@pytest.mark.parametrize("i8", [False, True])
def test_append_of_what_is_not_finite(i8):
    def spoil(table, kn, vn):
        kn[0, 1, 5], vn[3, 0, 9], kn[6, 0, 0], vn[7, 1, 2] = 0x7FC0, 0x7F80, 0xFF80, 0xFFC1

    _append_check(5, i8, 16, 64, 2, [2, 3, 4], [9, 3, 18], 2, spoil=spoil)


@pytest.mark.parametrize("i8", [False, True])
def test_append_of_zeros_and_extremes(i8):
    def spoil(table, kn, vn):
        kn[:2], vn[:2] = 0, 0x8000
        kn[2:4], vn[2:4] = 0x7F7F, 0x0001     # the largest and the smallest magnitude
        kn[4], vn[4] = 0x0080, 0xFF7F

    _append_check(6, i8, 16, 64, 1, [2, 2, 1, 1], [2, 5, 3, 17], 2, spoil=spoil)


@pytest.mark.parametrize("B, n", [(256, 1), (257, 2), (700, 40), (1, 3)])
def test_append_to_many_sequences(B, n):
    # more sequences than a workgroup asks for at once; fewer rows than pages they could need, and more
    g = np.random.default_rng(B)
    ns = (g.integers(1, n + 1, B) * (g.random(B) < 0.8)).tolist()
    _append_check(B, True, 16, 64, 1, ns, [int(x) for x in np.array(ns) + g.integers(0, 40, B)], 5, extra=2)


# ---- attention --------------------------------------------------------------------------------------


def _limits(out, lse, mag, smag, tokens, D):
    """What the roundings allow.  Scores: f32 sums of D exact products and two roundings of the
    scale, at most (D + 4) 2^-23 of scale * sum |q k| (the matrix unit may truncate, hence a whole
    step), over the keys that the row sees: ds.  A weight carries exp(2 ds), a bf16 rounding (2^-8) and the f32 exp and sums
    (tokens 2^-23); the result one more bf16 rounding."""
    ds = (D + 4) * 2.0**-23 * smag
    assert ds.max() < 2.0**-8, "scores too large to say anything"
    return (2.0**-8 + 2 * ds[..., None] + tokens * 2.0**-22) * mag + 2.0**-8 * np.abs(out) + 2.0**-126, ds + (tokens + 4) * 2.0**-23 + 2.0**-22 * np.abs(lse)


def _attend_check(seed, i8, P, D, H, R, ns, lens, max_pages, *, causal=True, spoil=None, qpad=0, extra=0, scale=None,
                  spare=2):
    g = syn.rng(60, seed)
    B = len(ns)
    pages = B * max_pages + spare
    k, v, ks, vs = _cache(g, pages, H, P, D, i8)
    table = _table(g, B, max_pages, pages)
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    T = int(off[-1]) + extra
    q = _rows(g, T, H * R, D)
    seen = (k.copy(), v.copy(), ks.copy(), vs.copy())  # what the definition reads
    if spoil:
        spoil(table, k, v, ks, vs, lens)
    wide = torch.full((T, H * R * D + qpad), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, : H * R * D] = bf16_dev(q).view(T, H * R * D)
    qd = wide[:, : H * R * D].unflatten(1, (H * R, D))
    out, lse = poison((T, H * R, D), torch.bfloat16), poison((T, H * R), torch.float32)
    untouched = host_bf16_bits(out)[int(off[-1]) :], host(lse)[int(off[-1]) :]
    c = wq.KvCache(*_devs(k, v, ks, vs))
    print(f"attention i8={i8} P={P} D={D} H={H} R={R} n={ns} lens={lens} causal={causal}", flush=True)
    wq.wq_kv_attention(c, qd, dev(off), dev(np.array(lens, np.int32)), dev(table), causal=causal, out=out, lse=lse, scale=scale)
    torch.cuda.synchronize()
    s = D**-0.5 if scale is None else scale
    want, want_lse, mag, smag = kvo.attention(*seen, q, off, lens, table, s, causal)
    got, got_lse = nm.bf16_to_f32(host_bf16_bits(out)).astype(np.float64), host(lse).astype(np.float64)
    n = int(off[-1])
    lim, lim_lse = _limits(want, np.where(np.isfinite(want_lse), want_lse, 0), mag, smag, max(max(lens), 1), D)
    empty = np.isneginf(want_lse[:n])
    assert np.array_equal(np.isneginf(got_lse[:n]), empty)
    assert not got[:n][empty].any()
    some = ~empty
    bad = np.argwhere(~(np.abs(got[:n] - want[:n]) <= lim[:n]))
    assert not len(bad), (len(bad), bad[:3].tolist(), got[tuple(bad[0])], want[tuple(bad[0])], lim[tuple(bad[0])])
    assert (np.abs(got_lse[:n][some] - want_lse[:n][some]) <= lim_lse[:n][some]).all()
    assert np.array_equal(host_bf16_bits(out)[n:], untouched[0]) and np.array_equal(host(lse)[n:], untouched[1])


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 48, 64, 128])
def test_attention_single_tokens(i8, D, P):
    _attend_check(P + D, i8, P, D, 2, 4, [1] * 9, [0, 1, 2, 15, 16, 17, 63, 65, 120], -(-128 // P))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("H, R", [(1, 1), (1, 16), (2, 5), (3, 3), (4, 8), (1, 40)])
def test_attention_head_groups(i8, H, R):
    _attend_check(H + R, i8, 32, 64, H, R, [1, 2, 5, 0, 1], [40, 97, 70, 12, 1], 4)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_prompts(i8, D, causal):
    _attend_check(D, i8, 32, D, 2, 2, [70, 33, 1, 130], [70, 150, 200, 131], 7, causal=causal, qpad=40, extra=3)


@pytest.mark.parametrize("i8", [False, True])
def test_attention_rows_that_see_nothing(i8):
    # more new rows than tokens (the first rows have negative positions), no tokens, a table too short
    for causal in (True, False):
        _attend_check(7, i8, 16, 64, 2, 2, [5, 4, 3, 20], [2, 0, -4, 60], 2, causal=causal)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("ns", [[1, 1, 3], [40, 20, 33]])
def test_attention_ignores_what_lies_behind_the_length(i8, ns):
    def spoil(table, k, v, ks, vs, lens):
        P = k.shape[2]
        used = np.zeros(len(k), bool)
        for b, length in enumerate(lens):
            for pg, page in enumerate(table[b]):
                keep = min(max(length - pg * P, 0), P)
                used[page] = keep > 0
                k[page, :, keep:], v[page, :, :, keep:] = (0x7F, 0xFF) if not i8 else (-128, 127)
        ks[~used], vs[~used] = 255, 255

    _attend_check(8, i8, 32, 128, 2, 2, ns, [41, 70, 96], 4, spoil=spoil)
    _attend_check(9, i8, 16, 64, 1, 4, ns, [41, 63, 33], 5, spoil=spoil, causal=False)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("ns", [[1, 1, 1], [50, 33, 20]])
def test_attention_skips_pages_that_are_none(i8, ns):
    def spoil(table, k, v, ks, vs, lens):
        table[0, 1], table[1, 0], table[2] = -1, len(k), (1 << 30)

    _attend_check(10, i8, 16, 64, 2, 2, ns, [50, 33, 40], 4, spoil=spoil)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("ns", [[1, 1], [3, 40]])
def test_attention_long_sequences(i8, ns):
    _attend_check(11, i8, 64, 64, 1, 4, ns, [3000, 1985], 47)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_sequences_in_many_and_in_few_parts(i8, D):
    # few items in parts of a step or two each; more items than an eighth of the runs
    _attend_check(13, i8, 64, D, 2, 3, [1, 40], [3000, 1985], 47, extra=2)
    _attend_check(14, i8, 64, D, 2, 3, [1] * 20, [60 * b + 5 for b in range(20)], 20)


@pytest.mark.parametrize("max_pages", [1, 18])
def test_attention_of_more_sequences_than_a_launch_plans(max_pages):
    # items, and runs that are cut, each in two launches
    g = np.random.default_rng(15)
    lens = [int(x) for x in g.integers(0, 65, 1100)]
    for b in (3, 1023, 1024, 1099):
        lens[b] = 64 * max_pages - b % 5
    _attend_check(15, True, 64, 64, 1, 1, [int(x) for x in g.integers(0, 2, 1100)], lens, max_pages)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_scales_and_scores_far_apart(D):
    # values' scales over forty powers of two between pages, a negative and a zero score scale
    def spoil(table, k, v, ks, vs, lens):
        pass

    for scale in (-0.02, 0.0, 0.3 / D):
        _attend_check(12, False, 16, D, 2, 2, [1, 30], [70, 90], 6, spoil=spoil, scale=scale)


@pytest.mark.parametrize("ns", [[2, 1], [40, 33]])
@pytest.mark.parametrize("i8", [False, True])
def test_a_page_marked_nan_reaches_only_rows_that_see_it(i8, ns):
    g = syn.rng(70, int(i8))
    P, D, H, R = 16, 64, 2, 2
    k, v, ks, vs = _cache(g, 12, H, P, D, i8)
    table, lens = _table(g, 2, 5, 12), np.array([75, 80], np.int32)
    vs[table[0, 4], 0] = 255      # tokens 64 .. of sequence 0, values of head 0
    ks[table[1, 4], 1] = 255      # tokens 64 .. of sequence 1, keys of head 1
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    q = _rows(g, int(off[-1]), H * R, D)
    out = wq.wq_kv_attention(wq.KvCache(*_devs(k, v, ks, vs)), bf16_dev(q), dev(off), dev(lens), dev(table))
    nan = np.isnan(nm.bf16_to_f32(host_bf16_bits(out))).all(-1)
    want = np.zeros_like(nan)
    for b in range(2):
        for i in range(ns[b]):
            want[off[b] + i, b * R : b * R + R] = lens[b] - ns[b] + i >= 64
    assert np.array_equal(nan, want) and np.array_equal(np.isnan(nm.bf16_to_f32(host_bf16_bits(out))).any(-1), want)


def test_cache_offsets_beyond_32_bits():
    # pages behind 4 GiB of codes: 70,000 pages of 64 KiB for each of k and v
    P, D, H, R, pages = 64, 128, 8, 2, 70000
    g = syn.rng(71)
    sizes = [(pages, H, P, D), (pages, H, D, P), (pages, H), (pages, H)]
    c = wq.KvCache(*(torch.empty(s, dtype=torch.uint8, device=DEV) for s in sizes))
    table = np.array([[69999, 3, 69000]], np.int32)
    kn, vn = _rows(g, 150, H, D), _rows(g, 150, H, D)
    off, lens = dev(np.array([0, 150], np.int64)), dev(np.array([150], np.int32))
    wq.wq_kv_append(c, bf16_dev(kn), bf16_dev(vn), off, lens, dev(table))
    small = [np.zeros((3, *s[1:]), np.uint8) for s in sizes]
    near = np.array([[0, 1, 2]], np.int32)
    kvo.append(*small, kn, vn, [0, 150], [150], near)
    at = torch.from_numpy(table[0].astype(np.int64)).to(DEV)
    for got, want in zip(c, small):
        got = host(got[at])
        for pg, keep in ((0, 64), (1, 64), (2, 22)):
            if want.ndim == 2:
                assert np.array_equal(got[pg], want[pg])
            elif want.shape[2] == P and want.shape[3] == D:
                assert np.array_equal(got[pg][:, :keep], want[pg][:, :keep])
            else:
                assert np.array_equal(got[pg][..., :keep], want[pg][..., :keep])
    q = _rows(g, 150, H * R, D)
    far = wq.wq_kv_attention(c, bf16_dev(q), off, lens, dev(table))
    close = wq.wq_kv_attention(wq.KvCache(*(t[at].contiguous() for t in c)), bf16_dev(q), off, lens, dev(near))
    assert np.array_equal(host_bf16_bits(far), host_bf16_bits(close))


# ---- as they are used ----------------------------------------------------------------------------------


def test_a_prompt_then_tokens_then_the_output_projection():
    """Rows appended in chunks and token by token, attention after each, and its output through
    the group quant and the grouped product: against the oracle, and eager against a graph."""
    g = syn.rng(72)
    P, D, H, R, B = 16, 128, 2, 4, 3
    steps = [[20, 5, 33], [1, 1, 1], [1, 1, 1], [3, 1, 0], [1, 1, 1]]
    max_pages = 4
    table = _table(g, B, max_pages, B * max_pages)
    c = wq.kv_cache(B * max_pages, H, P, D, device=DEV)
    ref = [host(t) for t in c]
    total = np.zeros(B, int)
    w8, ws, _ = (lambda p: (p[0], p[1], p[2]))(_fp8_weights(g, 2, 128, H * R * D // 2))
    for ns in steps:
        total += ns
        off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
        T = int(off[-1])
        kn, vn, q = _rows(g, T, H, D, 1.0), _rows(g, T, H, D, 1.0), _rows(g, T, H * R, D)
        offd, lensd, tabd = dev(off), dev(total.astype(np.int32)), dev(table)
        wq.wq_kv_append(c, bf16_dev(kn), bf16_dev(vn), offd, lensd, tabd)
        out, lse = wq.wq_kv_attention(c, bf16_dev(q), offd, lensd, tabd, return_lse=True)
        x8, _, st = wq.wq_group_quant_fp8_ue8m0(out.view(T, 2, -1))
        y = wq.wq_quant_matmul(x8, st, w8, ws, fp8_groups=2)
        torch.cuda.synchronize()
        kvo.append(*ref, kn, vn, off, total, table)
        for got, want in zip(c, ref):
            assert_same("cache", host(got), want)
        want, want_lse, mag, smag = kvo.attention(*ref, q, off, total, table, D**-0.5, True)
        lim, lim_lse = _limits(want, want_lse, mag, smag, int(total.max()), D)
        assert (np.abs(nm.bf16_to_f32(host_bf16_bits(out)) - want) <= lim).all()
        assert (np.abs(host(lse) - want_lse) <= lim_lse).all()
        # the projection reads what attention wrote, token by token
        again = wq.wq_quant_matmul(*(lambda a: (a[0], a[2]))(wq.wq_group_quant_fp8_ue8m0(out.clone().view(T, 2, -1))), w8, ws,
                                   fp8_groups=2)
        assert np.array_equal(host_bf16_bits(y), host_bf16_bits(again)) and np.isfinite(nm.bf16_to_f32(host_bf16_bits(y))).all()


def _fp8_weights(g, G, N, K):
    from oracle import fp8_group as fg

    w = nm.f64_to_bf16_rn(g.standard_normal((N, G, K)))
    q, _, e = fg.group_quant_fp8_packed(w)
    return dev(np.ascontiguousarray(q.transpose(1, 0, 2))), torch.full((G, N // 128, K // 128), 2.0**-9, device=DEV), e


def test_graphs_and_streams_share_nothing():
    """Two captured graphs over one long sequence each (their keys split over workgroups), and
    eager calls on two streams at once: each the same bytes as alone."""
    g = syn.rng(73)
    P, D, H, R, pages = 64, 128, 2, 4, 64
    sets = []
    for i in range(2):
        k, v, ks, vs = _cache(g, pages, H, P, D, True)
        c = wq.KvCache(*_devs(k, v, ks, vs))
        table, off = dev(_table(g, 1, pages, pages)), dev(np.array([0, 1], np.int64))
        lens = dev(np.array([4000 - 100 * i], np.int32))
        q = bf16_dev(_rows(g, 1, H * R, D))
        sets.append((c, q, off, lens, table))
    want = [host_bf16_bits(wq.wq_kv_attention(*s)) for s in sets]
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(wq.wq_kv_attention(*s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        for s, w in zip(sets, want):
            assert np.array_equal(host_bf16_bits(wq.wq_kv_attention(*s)), w)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert np.array_equal(host_bf16_bits(o), w)
    for _ in range(4):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(wq.wq_kv_attention(*s))
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert np.array_equal(host_bf16_bits(o), w)


def test_a_graph_follows_its_lengths():
    # one captured decode step (append, attend) replayed while the lengths in device memory grow
    g = syn.rng(74)
    P, D, H, R, B, max_pages = 16, 64, 2, 2, 3, 4
    table = _table(g, B, max_pages, B * max_pages)
    k, v, ks, vs = _cache(g, B * max_pages, H, P, D, False)
    c, e = wq.KvCache(*_devs(k, v, ks, vs)), wq.KvCache(*_devs(k, v, ks, vs))
    off, tab = dev(np.arange(B + 1, dtype=np.int64)), dev(table)
    lens = dev(np.array([0, 15, 40], np.int32))
    kn, vn, q = (torch.empty((B, n, D), dtype=torch.bfloat16, device=DEV) for n in (H, H, H * R))

    def step(cache):
        wq.wq_kv_append(cache, kn, vn, off, lens, tab)
        return wq.wq_kv_attention(cache, q, off, lens, tab, return_lse=True)

    graph, spare = torch.cuda.CUDAGraph(), wq.KvCache(*(t.clone() for t in c))
    for t in (kn, vn, q):
        t.copy_(bf16_dev(_rows(g, *t.shape)))
    step(spare)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = step(c)
    for _ in range(6):
        for t in (kn, vn, q):
            t.copy_(bf16_dev(_rows(g, *t.shape)))
        lens += 1
        graph.replay()
        want, want_lse = step(e)
        torch.cuda.synchronize()
        assert np.array_equal(host_bf16_bits(out), host_bf16_bits(want)) and np.array_equal(host(lse), host(want_lse))
        for a, b in zip(c, e):
            assert np.array_equal(host(a), host(b))
