"""Offsets that decrease, or lie outside 0 .. T, in attention behind a shared prefix (the reading of
them restated): the call's contract excludes them, and whatever they hold sequences have rows side by
side inside T, and every row that is joined has a join told by its sequence, whose places lie in the
workspace."""

import numpy as np
import pytest

import shared_plan as sp


def running(offsets, T):
    """First row of each sequence and their rows, as the plan reads them."""
    top = np.maximum.accumulate(np.clip(offsets, 0, T))
    return top, np.diff(top)


def as_given(offsets, T):
    """The same without the running maximum: each sequence's rows from its own offset on."""
    o = np.clip(offsets, 0, T)
    return o, np.maximum(np.diff(o), 0)


def places(row0, ns, group, R, D):
    """(row, place of it among its group's rows, the group's rows) of every row of a sequence in a group
    of more than one that has rows."""
    out, B = [], len(ns)
    lead = [0]
    for b in range(1, B):
        lead.append(b if group[b] < 0 or group[b] != group[b - 1] else lead[-1])
    for b in range(B):
        m = lead[b]
        mine = [x for x in range(B) if lead[x] == m and ns[x] > 0]
        if ns[b] and len(mine) > 1:
            end = max(row0[x] + ns[x] for x in mine)
            out += [(int(row0[b]) + i, (int(row0[b]) - int(row0[m])) * R + i * R, max(int(end - row0[m]), 0) * R) for i in range(ns[b])]
    return out


def batch(seed):
    g = np.random.default_rng(seed)
    B, T = int(g.integers(2, 14)), int(g.integers(1, 60))
    offsets = g.integers(-9, T + 20, B + 1)
    return g, B, T, offsets, np.cumsum(g.random(B) < 0.3).tolist()


def test_read_as_they_are_they_lead_outside():
    # what made the running maximum necessary: places before a group's first row (in 32 bits without a
    # sign, beyond all of them), and rows of several sequences
    wrong = [p for s in range(40) for _, B, T, o, group in [batch(s)] for p in places(*as_given(o, T), group, 4, 64)]
    assert any(at < 0 or at >= rows for _, at, rows in wrong)
    assert any(as_given(batch(s)[3], batch(s)[2])[1].sum() > batch(s)[2] for s in range(40))


@pytest.mark.parametrize("seed", range(40))
def test_rows_lie_side_by_side(seed):
    g, B, T, offsets, group = batch(seed)
    row0, ns = running(offsets, T)
    assert (ns >= 0).all() and ns.sum() == row0[-1] - row0[0] <= T
    assert all(0 <= at < rows for _, at, rows in places(row0, ns, group, 4, 64))
    # rows that the join goes over, offsets[0] to offsets[B]: each has one sequence
    of = [b for b in range(B) for _ in range(ns[b])]
    lo, hi = (int(np.clip(x, 0, T)) for x in (offsets[0], offsets[B]))
    assert row0[0] == lo and len(of) >= hi - lo
    # and the plan of those rows tells of each a join whose places are some run's, in its tile
    P, width, R, heads, D = 16, 40, 4, 2, int(g.choice([64, 256]))
    lens, shared = ([int(x) for x in g.integers(0, 600, B)] for _ in range(2))
    runs = 16
    taken, joins, _, _ = sp.plan([int(n) for n in ns], lens, group, shared, heads, R, D, P, width, runs, True)
    assert set(joins) == {(b, h, r) for b in range(B) for h in range(heads) for r in range(ns[b] * R)}
    for told in joins.values():
        for run, count, at in ([told[:3], told[3:6]] if told and len(told) > 3 else [told] if told else []):
            assert 0 <= run and run + count <= runs * sp.WAVES and 0 <= at < 256
