"""GPU parity of attention behind a shared prefix: against the definition in 64 bits within what its
roundings allow, for groups of any size, lengths, heads and masks; and as it is called."""

import ctypes

import numpy as np
import pytest
import torch

import kv_forms as kf
import shared_plan as sp
import synthetic as syn
from gpu_util import DEV, bf16_dev, dev, host, host_bf16_bits, poison
from oracle import numerics as nm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


def _limits(out, lse, mag, smag, tokens, D):
    """What the roundings allow.  Scores: f32 sums of D exact products and two roundings of the
    scale, at most (D + 4) 2^-23 of scale * sum |q k| (the matrix unit may truncate, hence a whole
    step): ds.  A weight carries exp(2 ds), a bf16 rounding (2^-8) and the f32 exp and sums (tokens
    2^-23, of which a step of 64 tokens makes no more than one part and its join's three roundings);
    the result one more bf16 rounding."""
    ds = (D + 4) * 2.0**-23 * smag
    assert ds.max() < 2.0**-8, "scores too large to say anything"
    lim = (2.0**-8 + 2 * ds[..., None] + (tokens + 64) * 2.0**-22) * mag + 2.0**-8 * np.abs(out) + 2.0**-126
    return lim, ds + (tokens + 64) * 2.0**-23 + 2.0**-22 * np.abs(lse)


def _inputs(seed, D, i8, ns, lens, group, shared, P, width, H, R, extra=2):
    """A cache, a table whose rows agree within a group where they say they do, queries."""
    g = syn.rng(120, seed, D, int(i8))
    B = len(ns)
    pages = B * width + 3
    c = list(kf.cache(g, pages, H, P, D, i8))
    table = g.permutation(pages)[: B * width].reshape(B, width).astype(np.int32)
    before = None  # the last sequence with rows of the group
    for b in range(B):
        if b and (group[b] < 0 or group[b] != group[b - 1]):
            before = None
        if ns[b] > 0:
            if before is not None:
                same = max(min(shared[b], width * P), 0) // P
                table[b, :same] = table[before, :same]
            before = b
    q = nm.f64_to_bf16_rn(g.standard_normal((sum(ns) + extra, H * R, D)))
    return c, table, q


def _check(c, table, q, ns, lens, group, shared, causal, *, scale=None, path=16, reads=None):
    B, (T, Hq, D) = len(ns), q.shape
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    n = int(off[-1])
    cd = wq.KvCache(*(dev(x) for x in c))
    args = [bf16_dev(q), dev(off), *(dev(np.array(x, np.int32)) for x in (lens, table, group, shared))]
    if path is not None:
        assert wq.wq_kv_attention_shared_path(cd, T, Hq, args[3]) == path
    out, lse = poison(q.shape, torch.bfloat16), poison((T, Hq), torch.float32)
    untouched = host_bf16_bits(out)[n:], host(lse).view(np.uint32)[n:]
    print(f"shared D={D} H={c[0].shape[1]} Hq={Hq} P={c[0].shape[2]} n={ns[:20]} lens={lens[:20]} group={group[:20]} shared={shared[:20]} causal={causal}", flush=True)
    wq.wq_kv_attention_shared(cd, *args, causal=causal, out=out, lse=lse, scale=scale)
    torch.cuda.synchronize()
    want, want_lse, mag, smag = kf.attention(reads or c, q, off, lens, table, D**-0.5 if scale is None else scale, causal)
    got, got_lse = nm.bf16_to_f32(host_bf16_bits(out)).astype(np.float64)[:n], host(lse).astype(np.float64)[:n]
    want, want_lse = want[:n], want_lse[:n]
    lost = np.isnan(want_lse)
    assert np.array_equal(np.isnan(got_lse), lost) and np.isnan(got[lost]).all()
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and not got[empty].any()
    some = np.isfinite(want_lse)
    lim, lim_lse = _limits(want, np.where(some, want_lse, 0), mag[:n], smag[:n], max(max(lens), 1), D)
    bad = np.argwhere(some[..., None] & ~(np.abs(got - want) <= lim))
    assert not len(bad), (len(bad), bad[:3].tolist(), got[tuple(bad[0])], want[tuple(bad[0])], lim[tuple(bad[0])])
    assert (np.abs(got_lse - want_lse)[some] <= lim_lse[some]).all()
    assert np.array_equal(host_bf16_bits(out)[n:], untouched[0]) and np.array_equal(host(lse).view(np.uint32)[n:], untouched[1])
    return cd, args, out, lse


CASES = {
    # eight answers to one question; two groups and one alone; many groups of different sizes; drafted
    # tokens; sequences without rows among them, in front of and behind a group; prompts behind a prefix
    "answers": dict(ns=[1] * 8, lens=[330, 321, 329, 350, 400, 322, 321, 333], group=[0] * 8, shared=[320] * 8, P=16, width=26, H=2, R=4),
    "groups": dict(ns=[1, 1, 1, 1, 1, 1], lens=[200, 140, 150, 77, 300, 290], group=[0, 0, 0, 7, 3, 3], shared=[128, 128, 128, 64, 256, 200], P=32, width=10, H=3, R=5),
    "one_row": dict(ns=[1, 1], lens=[129, 193], group=[0, 0], shared=[128, 128], P=64, width=4, H=1, R=1),
    "drafts": dict(ns=[4, 3, 4, 1, 2], lens=[700, 650, 641, 660, 1200], group=[0, 0, 0, 0, 0], shared=[640] * 5, P=64, width=20, H=2, R=8),
    "empty": dict(ns=[0, 1, 1, 0, 1, 0, 1, 1], lens=[5, 300, 290, 2, 270, 1, 200, 190], group=[0, 0, 0, 0, 0, 1, 1, 1], shared=[0, 256, 256, 0, 256, 0, 192, 190], P=32, width=10, H=2, R=4),
    "chunks": dict(ns=[12, 7, 12, 3], lens=[400, 340, 333, 360], group=[2, 2, 2, 2], shared=[320] * 4, P=16, width=26, H=2, R=4),
    "long": dict(ns=[1, 1, 1], lens=[9000, 8800, 8801], group=[0, 0, 0], shared=[8768] * 3, P=32, width=288, H=1, R=4),
    "wide": dict(ns=[1] * 40, lens=[300 + 7 * b for b in range(40)], group=[0] * 40, shared=[288] * 40, P=32, width=20, H=1, R=8),
    "uneven": dict(ns=[1, 1, 1, 1], lens=[500, 500, 500, 500], group=[0, 0, 0, 0], shared=[500, 333, 490, 500], P=16, width=32, H=2, R=4),
    "nothing": dict(ns=[1, 2, 1], lens=[60, 80, 70], group=[0, 0, 0], shared=[48, 48, 48], P=16, width=6, H=2, R=4),
}


def _case(name, D, i8, seed=1):
    f = dict(CASES[name])
    H, R, P, width = (f.pop(x) for x in ("H", "R", "P", "width"))
    return f, *_inputs(seed, D, i8, **f, P=P, width=width, H=H, R=R)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(CASES))
def test_groups(name, D, i8, causal):
    f, c, table, q = _case(name, D, i8)
    _check(c, table, q, **f, causal=causal)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    g = np.random.default_rng(900 + seed)
    ns, lens, group, shared, P, width = sp.batch(g, most=14, long=1500)
    D, H, R, i8 = int(g.choice([64, 128, 256])), int(g.integers(1, 5)), int(g.choice([1, 3, 4, 8])), bool(g.integers(2))
    ns = [min(n, max(1, 60 // R)) * (n > 0) for n in ns]
    c, table, q = _inputs(seed, D, i8, ns, lens, group, shared, P, width, H, R)
    # the tables agree from one sequence to the next as far as the second says: a group as far as its least
    _check(c, table, q, ns, lens, group, shared, bool(g.random() < 0.7), path=None)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_sequences_of_more_than_one_launch(D):
    # 1300 sequences in groups of 1 to 200, some across the border of two launches
    g = np.random.default_rng(30)
    B, P, width = 1300, 16, 12
    group = np.sort(g.integers(0, 25, B)).tolist()
    shared = [64 * (1 + x % 2) for x in group]
    lens = [int(s + x) for s, x in zip(shared, g.integers(1, 60, B))]
    ns = (g.random(B) < 0.9).astype(int).tolist()
    c, table, q = _inputs(31, D, True, ns, lens, group, shared, P, width, 1, 2)
    _check(c, table, q, ns, lens, group, shared, True)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_without_groups_it_is_attention(D, i8):
    f, c, table, q = _case("answers", D, i8)
    f.update(group=[-1] * 8)
    cd, args, out, lse = _check(c, table, q, **f, causal=True)
    want, want_lse = wq.wq_kv_attention(cd, *args[:4], return_lse=True)
    n = len(f["ns"])
    # the cut of the work differs, and with it the order of f32 sums of up to 400 tokens
    assert (lse[:n] - want_lse[:n]).abs().max() <= 2 * (400 + 64) * 2.0**-23 and want.shape == out.shape


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_to_a_sequence_take_their_own_tiles(D):
    f = dict(ns=[40, 20, 30], lens=[200, 180, 190], group=[0, 0, 0], shared=[128] * 3)
    c, table, q = _inputs(2, D, False, **f, P=16, width=14, H=2, R=4)
    _check(c, table, q, **f, causal=True, path=None)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("P", [48, 64])
@pytest.mark.parametrize("D, i8", [(64, True), (128, False), (128, True), (256, False)])
def test_row_tiles(D, i8, P, causal):
    # own tiles of 256 rows and a rest of 24, 104 and 132 (128, and rests of 24, 104 and 4, with heads of
    # 256); of the group 772 rows
    f = dict(ns=[70, 90, 33], lens=[300, 290, 250], group=[0, 0, 0], shared=[192] * 3)
    c, table, q = _inputs(4, D, i8, **f, P=P, width=7, H=2, R=4)
    _check(c, table, q, **f, causal=causal)


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_of_many_rows_are_attention_as_it_is(D):
    f = dict(ns=[520, 540], lens=[590, 600], group=[0, 0], shared=[48] * 2)
    c, table, q = _inputs(5, D, False, **f, P=16, width=38, H=1, R=4)
    cd, args, _, _ = _check(c, table, q, **f, causal=True, path=None)
    paths = [of(cd, *q.shape[:2], args[3]) for of in (wq.wq_kv_attention_shared_path, wq.wq_kv_attention_path)]
    assert paths[0] == paths[1] != 16


def _dense64(cd, q, ns, lens, table, scale):
    """kf.attention on the device, causal, of many tokens: (out, lse, mag, smag)."""
    k, v, ks, vs = cd
    P, (T, Hq, D) = k.shape[2], q.shape
    H = k.shape[1]
    value = lambda x: (x if x.dtype == torch.int8 else x.view(torch.float8_e4m3fn)).to(torch.float64)  # noqa: E731
    out, lse = torch.empty((T, Hq, D), dtype=torch.float64), torch.empty((T, Hq), dtype=torch.float64)
    mag, smag = torch.empty_like(out), torch.empty_like(lse)
    row = 0
    for n, length, pages in zip(ns, lens, dev(table).long()):
        pages = pages[: -(-length // P)]
        see = torch.arange(length, device=DEV)[None] <= (length - n + torch.arange(n, device=DEV))[:, None]
        for h in range(H):
            kk = (value(k[pages, h]) * torch.exp2(ks[pages, h].double() - 127)[:, None, None]).reshape(-1, D)[:length]
            vv = (value(v[pages, h]).transpose(1, 2) * torch.exp2(vs[pages, h].double() - 127)[:, None, None]).reshape(-1, D)[:length]
            at, rows = slice(h * (Hq // H), (h + 1) * (Hq // H)), slice(row, row + n)
            x = q[rows, at].double().reshape(-1, D)
            seen = see.repeat_interleave(Hq // H, 0)
            back = lambda y: y.view(n, Hq // H, *y.shape[1:]).cpu()  # noqa: E731
            smag[rows, at] = back(torch.where(seen, scale * (x.abs() @ kk.abs().T.contiguous()), 0.0).amax(1))
            s = torch.where(seen, scale * (x @ kk.T.contiguous()), -torch.inf)
            lse[rows, at] = back(torch.logsumexp(s, 1))
            w = torch.softmax(s, 1)
            out[rows, at], mag[rows, at] = back(w @ vv), back(w @ vv.abs())
        row += n
    return out.numpy(), lse.numpy(), mag.numpy(), smag.numpy()


@pytest.mark.parametrize("D, i8, P, S", [(128, False, 64, 18 * 8192), (128, True, 48, 65536), (64, False, 128, 18 * 8192), (64, True, 16, 65536),
                                         (256, False, 128, 5 * 16384), (256, True, 32, 32768)])
def test_runs_of_many_steps(D, i8, P, S):
    # more than 64 steps, or 64 groups of 16 tokens, in each of 256 runs: what tells pages is read 64 entries
    # at a time.  The cache is small: tables name its pages again and again.
    H, R, ns = 8, 2, [80, 100]
    g = syn.rng(121, D, P)
    c = list(kf.cache(g, 61, H, P, D, i8))
    shared = S // P * P
    lens = [shared + n + x for n, x in zip(ns, (3, 250))]
    table = g.integers(0, 61, (2, -(-max(lens) // P))).astype(np.int32)
    table[1, : shared // P] = table[0, : shared // P]
    q = nm.f64_to_bf16_rn(g.standard_normal((sum(ns), H * R, D)))
    cd = wq.KvCache(*(dev(x) for x in c))
    args = [bf16_dev(q), dev(np.array([0, 80, 180], np.int64)), *(dev(np.array(x, np.int32)) for x in (lens, table, [0, 0], [shared] * 2))]
    print(f"long runs D={D} i8={i8} P={P} tokens={lens}", flush=True)
    assert wq.wq_kv_attention_shared_path(cd, 180, H * R, args[3]) == 16
    out, lse = wq.wq_kv_attention_shared(cd, *args, return_lse=True)
    want, want_lse, mag, smag = _dense64(cd, args[0], ns, lens, table, D**-0.5)
    # sums of this many terms in f32: a step's 64 weights go into one sum, and there is one sum a step
    lim, lim_lse = _limits(want, want_lse, mag, smag, max(lens) // 64 + 64, D)
    got, got_lse = nm.bf16_to_f32(host_bf16_bits(out)), host(lse)
    assert (np.abs(got - want) <= lim).all() and (np.abs(got_lse - want_lse) <= lim_lse).all()


@pytest.mark.parametrize("falling", [False, True])
@pytest.mark.parametrize("ns", [[1] * 8, [20] * 8])
@pytest.mark.parametrize("D, i8", [(64, False), (128, False), (128, True), (256, True)])
def test_scores_that_climb_and_fall(D, i8, ns, falling):
    # the keys' scales double every second page, up to scores of 150 (of heads of 256, 113) or down from them: what weights are
    # relative to has to follow, by steps of any size, and rows whose scores are all below zero take part
    f = dict(ns=ns, lens=[900 + 3 * b for b in range(8)], group=[0] * 8, shared=[768] * 8)
    c, table, q = _inputs(6, D, i8, **f, P=32, width=30, H=1, R=4)
    order = np.arange(30)[::-1] if falling else np.arange(30)
    least = int(c[2].max())
    for b in range(8):
        c[2][table[b]] = (least - 15 + order // 2)[:, None]
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    smag = kf.attention(c, q, off, f["lens"], table, 1.0, True)[3]
    most = min(150.0, 0.9 * 2.0**15 / (D + 4))  # (_limits takes no larger ones)
    _check(c, table, q, **f, causal=True, scale=most / float(smag.max()))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 256])
def test_pages_marked_nan_and_rows_that_hold_one(D, i8):
    f, c, table, q = _case("groups", D, i8)
    c[2][table[0, 1], 0] = 255      # keys of head 0 in a page that group 0 shares
    c[3][table[1, 4], 1] = 255      # values of head 1 in a page of sequence 1 alone
    c[3][table[4, 6], 2] = 255      # of head 2, shared in group 3 for the most part
    q[3, 0, 5] = 0x7FC0
    for causal in (True, False):
        _check(c, table, q, **f, causal=causal)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_what_lies_behind_the_lengths_and_pages_that_are_none(D, i8):
    f, c, table, q = _case("drafts", D, i8)
    reads = [x.copy() for x in c]
    P = c[0].shape[2]
    for b, length in enumerate(f["lens"]):
        pg = length // P
        if length % P:
            c[0][table[b, pg], :, length % P :], c[1][table[b, pg], :, :, length % P :] = (-128, 127) if i8 else (0x7F, 0xFF)
        table[b, pg + 1 :] = 1 << 30
    table[:, 2] = -1                # a shared page that is none: its tokens are seen by nobody
    table[1, 10] = len(c[0])        # and one of a sequence's own
    _check(c, table, q, **f, causal=True, reads=reads)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales(D):
    f, c, table, q = _case("groups", D, False)
    for scale in (-0.02, 0.0, 0.3 / D):
        _check(c, table, q, **f, causal=True, scale=scale)


def test_a_sequence_that_sees_less_than_its_group():
    # shared numbers beyond what a row sees, beyond the table, negative, and of single members: never more
    # than all rows see is taken for all
    f = dict(ns=[2, 5, 1, 1], lens=[130, 131, 300, 500], group=[0, 0, 0, 0], shared=[1 << 30, 400, 256, 2147483647])
    c, table, q = _inputs(3, 128, True, **f, P=16, width=20, H=2, R=2)
    table[1:, :19] = table[0, :19]
    for causal in (True, False):
        _check(c, table, q, **f, causal=causal)
    f.update(shared=[128, -5, 128, 128])
    _check(c, table, q, **f, causal=True)


def _bits(out, lse, n):
    return host_bf16_bits(out)[:n], host(lse).view(np.uint32)[:n]


def _same(a, b):
    return all(np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", ["answers", "drafts", "empty", "long"])
def test_workspaces(name, D, i8):
    f, c, table, q = _case(name, D, i8)
    n = sum(f["ns"])
    cd, args, out, lse = _check(c, table, q, **f, causal=True)
    want = _bits(out, lse, n)
    T, heads, _ = q.shape
    pages, H, P, _ = c[0].shape
    d = wq.KvCacheDesc(wq.WQ_KV_INT8 if i8 else wq.WQ_KV_E4M3, pages, H, P, D, *(t.data_ptr() for t in cd), args[3].data_ptr(),
                       table.shape[1], table.shape[1])
    ctx = wq.context(DEV).handle
    need = wq.lib().wq_kv_attention_shared_workspace_bytes(ctx, ctypes.byref(d), T, heads, len(f["ns"]))
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    for at, size in ((ws.data_ptr(), need), (None, 0)):
        out, lse = poison(q.shape, torch.bfloat16), poison((T, heads), torch.float32)
        assert wq.lib().wq_kv_attention_shared(
            ctx, ctypes.byref(d), args[0].data_ptr(), heads * D, T, heads, len(f["ns"]), args[1].data_ptr(), args[2].data_ptr(),
            args[4].data_ptr(), args[5].data_ptr(), D**-0.5, 1, out.data_ptr(), heads * D, lse.data_ptr(), at, size,
            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert _same(_bits(out, lse, n), want)
    assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("name, D, i8", [("answers", 128, False), ("groups", 64, True), ("drafts", 256, False), ("long", 128, True)])
def test_graphs_with_eager_calls_between(name, D, i8):
    f, c, table, q = _case(name, D, i8)
    cd, args, _, _ = _check(c, table, q, **f, causal=True)
    n = sum(f["ns"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = wq.wq_kv_attention_shared(cd, *args, return_lse=True)
    g = np.random.default_rng(1)
    for i in range(4):
        args[0].copy_(bf16_dev(nm.f64_to_bf16_rn(g.standard_normal(q.shape))))
        if i:  # shorter sequences that share less: the plan follows them
            args[2].copy_((args[2] - int(g.integers(0, 20))).clamp(min=0))
            args[5].copy_((args[5] - int(g.integers(0, 40))).clamp(min=0))
        if i == 3:
            args[4].copy_(torch.arange(len(args[4]), device=DEV) // 2)
        graph.replay()
        eager = wq.wq_kv_attention_shared(cd, *args, return_lse=True)
        torch.cuda.synchronize()
        assert _same(_bits(out, lse, n), _bits(*eager, n))


@pytest.mark.parametrize("D", [64, 256])
def test_two_streams_at_once(D):
    sets = []
    for i, name in enumerate(("drafts", "wide")):
        f, c, table, q = _case(name, D, bool(i))
        cd, args, out, lse = _check(c, table, q, **f, causal=True)
        sets.append((cd, args, _bits(out, lse, sum(f["ns"]))))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for st, (cd, args, _) in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(wq.wq_kv_attention_shared(cd, *args, return_lse=True))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        want = sets[i % 2][2]
        assert _same(_bits(*o, len(want[0])), want)
