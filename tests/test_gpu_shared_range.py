"""Attention behind a shared prefix where its weights' size and rounding tell: scores that climb by
less than what moves the weights' base, at values whose weighted sums come near 2^120; rows of one
token, of one large weight and of a few."""

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from gpu_util import bf16_dev, dev, host, host_bf16_bits
from oracle import numerics as nm
from test_gpu_shared import _limits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


def _attend(c, table, q, ns, lens, group, shared, scale=None):
    """(out bits, lse) of causal attention, within what its roundings allow of the definition in 64 bits.

    The quotient's line is the sum of the weights as they are rounded for the other: with e the relative
    rounding of each and w the exact weights it is sum w (1 + e) v / sum w (1 + e), off by sum w e (v - out) in
    the first order, e below 2^-8: by 2^-8 (sum w |v| + |out|) at most and 2^-7 of that in the second."""
    T, Hq, D = q.shape
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    cd = wq.KvCache(*(dev(x) for x in c))
    args = [bf16_dev(q), dev(off), *(dev(np.array(x, np.int32)) for x in (lens, table, group, shared))]
    assert wq.wq_kv_attention_shared_path(cd, T, Hq, args[3]) == 16
    print(f"shared D={D} {c[0].dtype} H={c[0].shape[1]} Hq={Hq} n={ns[:20]} lens={lens[:20]} group={group[:20]}", flush=True)
    out, lse = wq.wq_kv_attention_shared(cd, *args, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    want, want_lse, mag, smag = kf.attention(c, q, off, lens, table, D**-0.5 if scale is None else scale, True)
    bits, lse = host_bf16_bits(out), host(lse)
    lim, lim_lse = _limits(want, want_lse, mag, smag, max(lens), D)
    lim += (2.0**-8 + 2.0**-14) * np.abs(want) + 2.0**-14 * mag
    bad = np.argwhere(~(np.abs(nm.bf16_to_f32(bits).astype(np.float64) - want) <= lim))
    assert not len(bad), (len(bad), bad[:3].tolist())
    assert (np.abs(lse - want_lse) <= lim_lse).all()
    return bits, lse

# code and key scale byte of a score, in powers of two with q = 1 and the scale ln 2
CLIMBS = {
    False: {9.0: (0x51, 127), 11.0: (0x53, 127), 24.0: (0x5C, 127)},
    True: {8.5: (17, 126), 11.5: (23, 126), 40.5: (81, 126)},
}
STEPS = 6  # of 64 tokens


def _ladder(D, i8, climb, value, ns, own=50, group=0, H=1, R=8, P=64, seed=1):
    """Sequences behind STEPS steps of tokens whose scores are zero but for one token of each second
    step, which has `climb` (times q's first element) and the values `value`
    (code, byte); the other tokens of these pages have small codes at the same scale."""
    g = syn.rng(130, seed, D, int(i8))
    B, S = len(ns), 64 * STEPS
    lens = [S + own + n for n in ns]
    width = -(-max(lens) // P)
    pages = B * width + 3
    k, v, ks, vs = kf.cache(g, pages, H, P, D, i8)
    code, kbyte = CLIMBS[i8][climb]
    k[:], ks[:] = 0, kbyte
    v[:] = g.integers(-3, 4, v.shape) if i8 else g.integers(0, 0x20, v.shape)
    vs[:] = value[1]
    table = g.permutation(pages)[: B * width].reshape(B, width).astype(np.int32)
    table[1:, : S // P] = table[0, : S // P]
    if group < 0:  # (each sequence has steps of its own then, the same ones)
        table[:] = table[0]
    for step, at in zip(range(1, STEPS, 2), (0, 37, 63)):
        page, slot = table[0, (64 * step + at) // P], (64 * step + at) % P
        k[page, :, slot, 0] = code
        v[page, :, :, slot] = np.array(value[0]).astype(v.dtype)
    q = np.zeros((sum(ns), H * R, D))
    q[..., 0] = g.choice([1.0, 0.96875, 0.875, 0.75, 0.5, 0.0, -1.0], q.shape[:2])
    q[0, 0, 0] = 1.0
    f = dict(ns=ns, lens=lens, group=[group] * B, shared=[S] * B)
    return f, [k, v, ks, vs], table, nm.f64_to_bf16_rn(q)


@pytest.mark.parametrize("ns, group", [([1] * 8, 0), ([20] * 4, 0), ([20] * 2, -1)])
@pytest.mark.parametrize("D, i8, climb", [(D, i8, x) for D in (64, 128, 256) for i8 in (False, True) for x in CLIMBS[i8]])
def test_values_whose_weighted_sums_come_near_the_bound(D, i8, climb, ns, group):
    # values of 2^118, three of which are the most that a row's sum holds at weights up to 1: below 2^120,
    # what the call allows.  At weights of 2^11 one of them is infinite in 32 bits.
    value = (64, 239) if i8 else (0x78, 237)  # 2^6 2^112, 2^8 2^110
    f, c, table, q = _ladder(D, i8, climb, value, ns, group=group)
    bits, _ = _attend(c, table, q, **f, scale=float(np.log(2.0)))
    assert np.isfinite(nm.bf16_to_f32(bits)).all()


def _value_rows(c, table, i8, pos, P):
    """bf16 values of every sequence's token pos[b], all heads: [B, H, D], exact."""
    page, slot = table[np.arange(len(pos)), pos // P], pos % P
    codes = kf.kvo.decode(c[1][page, :, :, slot])
    return nm.f64_to_bf16_rn(codes * 2.0 ** (c[3][page].astype(np.float64) - 127)[..., None])


@pytest.mark.parametrize("group", [0, -1])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_see_one_token_are_its_value(D, i8, group):
    # The one weight is a power of two times anything in (1/2, 1]; its rounding to bf16 stands above and below
    # the line of the quotient, which leaves a few roundings of f32 around a value that bf16 holds: the value.
    P, H, R, ns = 32, 2, 24, [3, 5, 2]
    f = dict(ns=ns, lens=ns, group=[group] * 3, shared=[0] * 3)
    g = syn.rng(131, D, int(i8))
    c = list(kf.cache(g, 9, H, P, D, i8))
    table = g.permutation(9).reshape(3, 3).astype(np.int32)
    q = nm.f64_to_bf16_rn(g.standard_normal((sum(ns), H * R, D)))
    bits, _ = _attend(c, table, q, **f)
    first = np.concatenate(([0], np.cumsum(ns)))[:-1]
    want = np.repeat(_value_rows(c, table, i8, np.zeros(3, int), P), R, axis=1)
    # (as numbers: a value of -0 added to the accumulators' 0 is 0)
    assert np.array_equal(nm.bf16_to_f32(bits[first]), nm.bf16_to_f32(want))


@pytest.mark.parametrize("ns", [[1] * 8, [20] * 4])
@pytest.mark.parametrize("D, i8", [(64, True), (128, False), (128, True), (256, True)])
def test_one_token_far_above_the_others_gives_its_value(D, i8, ns):
    # scores 24 (E4M3) or 40.5 above all others', times numbers from 7/8 on: the others weigh at most 2^-21
    # each, 2^-12 all 440 together, and their values are no larger than the one's, which bf16 holds and
    # whose half step is 2^-9 of it or more
    climb = 40.5 if i8 else 24.0
    f, c, table, q = _ladder(D, i8, climb, (64, 130) if i8 else (0x51, 127), ns)
    q[:] = 0
    g = np.random.default_rng(3)
    q[..., 0] = nm.f64_to_bf16_rn(g.choice([1.0, 0.9921875, 0.96875, 0.9375, 0.90625, 0.875], q.shape[:2]))
    bits, _ = _attend(c, table, q, **f, scale=float(np.log(2.0)))
    assert (bits == nm.f64_to_bf16_rn(np.array(64.0 * 8 if i8 else 9.0))).all()


@pytest.mark.parametrize("ns", [[1] * 16, [40] * 2])
@pytest.mark.parametrize("D, i8", [(64, False), (128, False), (128, True), (256, False)])
def test_errors_are_those_of_independent_roundings(D, i8, ns):
    # Rows of a few large weights.  Each weight's rounding is off by e (relative), at most 2^-8 and uniform for
    # a mantissa m within 2^-8 / m: mean square 2^-16 / 3 E[1 / m^2], of mantissas spread over their logarithm
    # (1 - 1/4) / (2 ln 2) = 0.541.  The quotient is over the rounded weights, so that an output is off by
    # sum w e (v - out), with w the exact weights, and its own rounding, half a step at most and
    # uniform.  Both in the mean square over all outputs, with 15 % for the sample (thousands of weights;
    # a common error of numerator or denominator would add 40 % and more).
    H, R, P, S = 2, 8, 32, 512
    g = syn.rng(132, D, int(i8), len(ns))
    B = len(ns)
    lens = [S + 40 + n for n in ns]
    width = -(-max(lens) // P)
    c = list(kf.cache(g, B * width + 3, H, P, D, i8))
    c[2][:], c[3][:] = (120, 120) if i8 else (126, 126)
    table = g.permutation(len(c[0]))[: B * width].reshape(B, width).astype(np.int32)
    table[1:, : S // P] = table[0, : S // P]
    q = nm.f64_to_bf16_rn(g.standard_normal((sum(ns), H * R, D)))
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    spread = kf.attention(c, q, off, lens, table, 1.0, True)[3].max()
    scale = 100.0 / spread
    bits, _ = _attend(c, table, q, ns, lens, [0] * B, [S] * B, scale)
    got = nm.bf16_to_f32(bits).astype(np.float64)
    qf = nm.bf16_to_f32(q).astype(np.float64)
    error, allowed, most = 0.0, 0.0, []
    for b in range(B):
        pos = np.arange(lens[b])
        for h in range(H):
            k = kf.kvo.decode(c[0][table[b, pos // P], h, pos % P]) * 2.0 ** (int(c[2][0, 0]) - 127)
            v = kf.kvo.decode(c[1][table[b, pos // P], h, :, pos % P]) * 2.0 ** (int(c[3][0, 0]) - 127)
            for i in range(ns[b]):
                for r in range(h * R, h * R + R):
                    s = scale * (k[: lens[b] - ns[b] + i + 1] @ qf[off[b] + i, r])
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    want = w @ v[: len(w)]
                    most.append(w.max())
                    error += np.square(got[off[b] + i, r] - want).sum()
                    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0**-100))) - 8)
                    allowed += np.square(half).sum() / 3 + 0.541 * 2.0**-16 / 3 * (np.square(w) @ np.square(v[: len(w)] - want)).sum()
    assert np.mean(most) > 0.4, "rows of a few large weights"
    assert error <= 1.15**2 * allowed, (error / allowed) ** 0.5


@pytest.mark.parametrize("ns", [[1] * 8, [20] * 4])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_without_groups_outputs_are_those_of_attention(D, i8, ns):
    # each within what its roundings allow of the definition: both weights' (2^-8 of sum w |v|, and of |out| where
    # the sum is of rounded ones) and both outputs' (2^-8), and the f32 sums of either
    H, R, P, width = 2, 4, 16, 26
    g = syn.rng(134, D, int(i8), len(ns))
    B = len(ns)
    lens = [300 + 13 * b for b in range(B)]
    c = kf.cache(g, B * width, H, P, D, i8)
    table = g.permutation(B * width).reshape(B, width).astype(np.int32)
    q = nm.f64_to_bf16_rn(g.standard_normal((sum(ns), H * R, D)))
    off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
    cd = wq.KvCache(*(dev(x) for x in c))
    args = [bf16_dev(q), dev(off), dev(np.array(lens, np.int32)), dev(table)]
    ids, none = (dev(np.full(B, x, np.int32)) for x in (-1, 0))
    assert wq.wq_kv_attention_shared_path(cd, *q.shape[:2], args[3]) == 16
    got, got_lse = wq.wq_kv_attention_shared(cd, *args, ids, none, return_lse=True)
    ref, ref_lse = wq.wq_kv_attention(cd, *args, return_lse=True)
    want, want_lse, mag, smag = kf.attention(c, q, off, lens, table, D**-0.5, True)
    lim, lim_lse = _limits(want, want_lse, mag, smag, max(lens), D)
    a, b = (nm.bf16_to_f32(host_bf16_bits(x)).astype(np.float64) for x in (got, ref))
    assert (np.abs(a - b) <= 2 * lim + (2.0**-8 + 2.0**-14) * np.abs(want) + 2.0**-14 * mag).all()
    assert (np.abs(host(got_lse) - host(ref_lse)) <= 2 * lim_lse).all()
