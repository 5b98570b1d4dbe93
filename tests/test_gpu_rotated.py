"""GPU parity of rows appended with turned keys, and of turned queries: codes, scales and queries bit
for bit against the oracle, and as the call is made: in place, in wider rows, captured."""

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from gpu_util import DEV, assert_same, bf16_dev, dev, host, host_bf16_bits, poison
from oracle import layer
from oracle import numerics as nm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


def _angles(positions, rot):
    i = np.arange(rot // 2)
    turn = np.arange(positions)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return np.stack((np.cos(turn), np.sin(turn)), 1).astype(np.float32)


def _rows(g, T, H, D, loud=0.0):
    return nm.f64_to_bf16_rn(g.standard_normal((T, H, D)) * np.exp2(loud * g.standard_normal((T, 1, 1))))


def _one_nan(bits):
    return np.where((bits & 0x7FFF) > 0x7F80, 0x7FC0, bits).astype(np.uint16)


def _check(seed, i8, P, D, H, R, rot, pairs, ns, lens, max_pages, *, loud=2.0, spoil=None, pad=0, extra=0, positions=None, with_q=True):
    g = syn.rng(110, seed)
    B = len(ns)
    pages = B * max_pages + 2
    c = list(kf.cache(g, pages, H, P, D, i8))
    table = g.permutation(pages)[: B * max_pages].reshape(B, max_pages).astype(np.int32)
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    T, n = int(off[-1]) + extra, int(off[-1])
    kn, vn, q = _rows(g, T, H, D, loud), _rows(g, T, H, D, loud), _rows(g, T, H * R, D)
    angles = _angles(max(*lens, 1) if positions is None else positions, rot)
    if spoil:
        spoil(table, kn, vn, q, angles)
    cd = wq.KvCache(*(dev(a) for a in c))

    def wide(bits):
        t = torch.full((T, bits.shape[1] * D + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
        t[:, : bits.shape[1] * D] = bf16_dev(bits).view(T, -1)
        return t[:, : bits.shape[1] * D].unflatten(1, (bits.shape[1], D))

    kd, vd, qd = wide(kn), wide(vn), wide(q)
    out = poison((T, H * R * D + pad), torch.bfloat16)
    before = host(out.view(torch.int16))
    qo = out[:, : H * R * D].unflatten(1, (H * R, D))
    args = (cd, kd, vd, dev(off), dev(np.array(lens, np.int32)), dev(table), dev(angles))
    kw = dict(q=qd, q_out=qo) if with_q else {}
    print(f"rotated i8={i8} P={P} D={D} H={H} R={R} rot={rot} pairs={pairs} n={ns} lens={lens}", flush=True)
    wq.wq_kv_append_rotated(*args, interleaved=pairs, **kw)
    torch.cuda.synchronize()
    layer.append_rotated(*c, kn, vn, angles, pairs, off, lens, table)
    for twice in (False, True):
        for name, got, want in zip(("k", "v", "k_scale", "v_scale"), cd, c):
            assert_same(name + (" again" if twice else ""), host(got), want)
        if not twice:  # the same call again writes the same bytes
            wq.wq_kv_append_rotated(*args, interleaved=pairs, **kw)
            torch.cuda.synchronize()
    after = host(out.view(torch.int16))
    if not with_q:
        assert np.array_equal(after, before)
        return
    y = layer.turned(nm.bf16_to_f32(q[:n]), layer.positions_of(off, lens), angles, pairs)
    want = np.where(np.isnan(y), 0x7FC0, nm.f64_to_bf16_rn(np.where(np.isfinite(y), y, 0.0).astype(np.float64)))
    want = np.where(np.isposinf(y), 0x7F80, np.where(np.isneginf(y), 0xFF80, want)).astype(np.uint16)
    assert_same("q", _one_nan(host_bf16_bits(qo)[:n]), _one_nan(want))
    assert np.array_equal(after[n:], before[n:]) and np.array_equal(after[:, H * R * D :], before[:, H * R * D :])
    # in place, the queries alone differing
    wq.wq_kv_append_rotated(*args, interleaved=pairs, q=qd, q_out=qd)
    assert np.array_equal(_one_nan(host_bf16_bits(qd)[:n]), _one_nan(want)) and np.array_equal(host_bf16_bits(qd)[n:], q[n:])


@pytest.mark.parametrize("i8, pairs", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("P", [16, 48, 64, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths(i8, pairs, P, D):
    # one row at a page's start, inside, at its end; runs over a border; whole pages; nothing
    _check(P + D, i8, P, D, 2, 2, D, pairs, [1, 1, 1, 0, 3, P, P + 5, 2 * P + 1], [1, 2, P, 9, P + 1, P, 2 * P + 2, 2 * P + 1], 3)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D, rot", [(64, 16), (64, 48), (128, 32), (128, 112), (256, 64), (256, 240)])
def test_parts_of_a_head(D, rot, pairs):
    _check(rot, D == 128, 32, D, 3, 2, rot, pairs, [4, 1, 40], [30, 33, 41], 2, pad=24, extra=3)


@pytest.mark.parametrize("H, R", [(1, 1), (1, 16), (3, 5), (8, 4), (5, 3)])
def test_heads(H, R):
    for ns in ([1, 1, 1], [30, 2, 50]):
        _check(H + R, False, 32, 128, H, R, 128, False, ns, [30, 31, 60], 2, extra=2)


# a page's queries by one workgroup or several, whole fours of heads and rests of them
@pytest.mark.parametrize("P, D, H, R", [(128, 256, 1, 16), (256, 128, 2, 5), (64, 128, 1, 70), (256, 64, 3, 1), (48, 256, 2, 6)])
def test_prompts_of_many_heads(P, D, H, R):
    for pairs in (False, True):
        _check(P + R, pairs, P, D, H, R, D // 2, pairs, [P + 40, 2, P - 7], [P + 43, P + 1, P - 7], 3, extra=5)


@pytest.mark.parametrize("i8", [False, True])
def test_without_queries(i8):
    _check(1, i8, 16, 64, 2, 2, 64, False, [1, 20, 0], [5, 33, 9], 4, with_q=False)


@pytest.mark.parametrize("i8", [False, True])
def test_rows_much_larger_and_much_smaller(i8):
    for seed, loud in ((1, 12.0), (2, 0.0)):
        _check(seed, i8, 64, 128, 2, 1, 128, False, [1] * 12 + [5], list(range(7, 19)) + [64], 2, loud=loud)


@pytest.mark.parametrize("ns", [[20, 7, 5, 4], [1, 1, 1, 1]])
@pytest.mark.parametrize("i8", [False, True])
def test_beyond_the_table_and_before_the_first_token(i8, ns):
    _check(3, i8, 16, 64, 2, 2, 32, True, ns, [37, 3, 0, -2], 2)


@pytest.mark.parametrize("ns", [[20, 20, 3], [1, 1, 2]])
@pytest.mark.parametrize("i8", [False, True])
def test_pages_that_are_none(i8, ns):
    def spoil(table, kn, vn, q, angles):
        table[0, 0], table[1, 1], table[2, 0] = -1, 1 << 30, len(table) * 2 + 2

    _check(4, i8, 16, 64, 2, 2, 64, False, ns, [20, 25, 3], 2, spoil=spoil)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("i8", [False, True])
def test_positions_without_angles(i8, pairs):
    _check(5, i8, 16, 64, 2, 2, 32, pairs, [2, 20, 1, 1], [9, 30, 12, 13], 2, positions=12)


@pytest.mark.parametrize("i8", [False, True])
def test_what_is_not_finite_and_the_extremes(i8):
    def spoil(table, kn, vn, q, angles):
        kn[0, 1, 5], vn[3, 0, 9], kn[6, 0, 0], vn[7, 1, 2], q[2, 0, 1], q[3, 1, 40] = 0x7FC0, 0x7F80, 0xFF80, 0xFFC1, 0x7F80, 0x7FC0
        kn[1, 0, :] = 0x7F7F   # a pair's sum beyond the largest number
        kn[4], vn[4] = 0, 0x8000
        kn[5], vn[5] = 0x0001, 0x0001
        angles[3, 0, 2], angles[8, 1, 0] = np.nan, np.inf

    with np.errstate(over="ignore"):
        _check(6, i8, 16, 64, 2, 2, 64, False, [2, 3, 4], [9, 3, 18], 2, spoil=spoil)


@pytest.mark.parametrize("B, n", [(256, 1), (257, 2), (700, 40), (1, 3)])
def test_many_sequences(B, n):
    g = np.random.default_rng(B)
    ns = (g.integers(1, n + 1, B) * (g.random(B) < 0.8)).tolist()
    _check(B, True, 16, 64, 1, 2, 64, False, ns, [int(x) for x in np.array(ns) + g.integers(0, 40, B)], 5, extra=2)


def test_far_positions():
    # one long sequence: four tokens at its end, angles of positions up to 131071
    _check(7, False, 128, 64, 1, 2, 64, False, [4], [131072], 1024)


def test_unturned_it_is_append():
    g = syn.rng(111)
    f, c, table, _ = kf.inputs("items64", 128, True, 5)
    T = int(f["offsets"][-1])
    kn, vn = bf16_dev(_rows(g, T, f["H"], 128, 1.0)), bf16_dev(_rows(g, T, f["H"], 128, 1.0))
    a, b = (wq.KvCache(*(dev(x) for x in c)) for _ in range(2))
    rest = dev(f["offsets"]), dev(np.array(f["lens"], np.int32)), dev(table)
    angles = torch.zeros((256, 2, 64), device=DEV)
    angles[:, 0] = 1.0
    wq.wq_kv_append(a, kn, vn, *rest)
    wq.wq_kv_append_rotated(b, kn, vn, *rest, angles)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_it_follows_its_lengths():
    g = syn.rng(112)
    P, D, H, R, B, width = 16, 64, 2, 2, 3, 4
    table = dev(g.permutation(B * width).reshape(B, width).astype(np.int32))
    c = wq.KvCache(*(dev(x) for x in kf.cache(g, B * width, H, P, D, False)))
    e = wq.KvCache(*(t.clone() for t in c))
    off, lens = dev(np.arange(B + 1, dtype=np.int64)), dev(np.array([0, 15, 40], np.int32))
    angles = wq.rotary_angles(64, 32, device=DEV)
    kn, vn, q = (torch.empty((B, n, D), dtype=torch.bfloat16, device=DEV) for n in (H, H, H * R))

    def step(cache):
        return wq.wq_kv_append_rotated(cache, kn, vn, off, lens, table, angles, q=q)

    step(wq.KvCache(*(t.clone() for t in c)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c)
    for _ in range(6):
        for t in (kn, vn, q):
            t.copy_(bf16_dev(_rows(g, *t.shape)))
        lens += 1
        graph.replay()
        want = step(e)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(x, y) for x, y in zip(c, e))
