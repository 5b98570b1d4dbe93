"""Attention behind a shared prefix at the edge of the values' range: scores that climb by less than
what moves the weights' base, at values whose weighted sums come near 2^120."""

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from oracle import numerics as nm
from test_gpu_shared import _check

pytestmark = pytest.mark.gpu

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
    _, _, out, _ = _check(c, table, q, **f, causal=True, scale=float(np.log(2.0)))
    assert torch.isfinite(out[: sum(ns)].float()).all()
