"""The runs of attention behind a shared prefix (restated): every step of every item once, parts in
slots of their own, each row's join told as its parts lie, whatever lengths, groups and numbers of
shared tokens are given."""

import numpy as np
import pytest

import shared_plan as sp


@pytest.mark.parametrize("seed", range(120))
def test_runs_cover_the_work(seed):
    g = np.random.default_rng(700 + seed)
    ns, lens, group, shared, P, width = sp.batch(g)
    D, heads, R = int(g.choice([64, 256])), int(g.integers(1, 6)), int(g.choice([1, 4, 5, 16]))
    causal = bool(g.random() < 0.7)
    runs = int(g.choice([2, 3, 7, 64, 256]))
    taken, joins, sh, holder = sp.plan(ns, lens, group, shared, heads, R, D, P, width, runs, causal)
    row0 = np.concatenate(([0], np.cumsum(ns)))
    slots = set()
    for (of_group, b, h, tile), parts in taken.items():
        # steps in order, each once; the first part holds step 0; the others are of runs of their own
        assert [p[1] for p in parts] == [0] + [p[2] for p in parts[:-1]] and parts[-1][2] == parts[-1][5]
        assert [p[0] for p in parts] == list(range(parts[0][0], parts[0][0] + len(parts)))
        for i, (run, lo, hi, kind, axis, _) in enumerate(parts):
            assert (kind == "run") == (i > 0) and (kind == "out") <= (len(parts) == 1)
            if kind == "run":
                assert (axis, run) not in slots and run < runs * (sp.WAVES if axis == sp.NARROW else 1)
                slots.add((axis, run))
    # items: all of them
    size = [sp.kind_of(n * R, D)[1] for n in ns]
    own = {(b, h, t) for b in range(len(ns)) for h in range(heads) for t in range(-(-ns[b] * R // size[b]))}
    assert {k[1:4] for k in taken if not k[0]} == own
    for b in range(len(ns)):
        if sh[b] and ns[b]:
            assert ns[holder[b]] > 0 and group[holder[b]] == group[b] >= 0
            assert sh[b] * sp.TILE <= min(shared[b], width * P) // P * P and sh[b] * sp.TILE <= max(lens[b] - ns[b] * causal, 0)
    # joins
    for b in range(len(ns)):
        for h in range(heads):
            for r in range(ns[b] * R):
                told, mine = joins[(b, h, r)], taken[(False, b, h, r // size[b])]
                if told is None:
                    assert sh[b] == 0 and [p[3] for p in mine] == ["out"]
                    continue
                assert told[:3] == (mine[0][0], len(mine), r % size[b]) and len(told) == (7 if sh[b] else 3)
                if sh[b]:
                    parts, m = taken[told[6]], told[6][1]
                    rows = sum(ns[x] for x in range(m, len(ns)) if all(group[y] == group[m] for y in range(m, x + 1)))
                    tile = sp.kind_of(rows * R, D)[1]
                    assert told[3:5] == (parts[0][0], len(parts)) and (row0[b] - row0[m]) * R + r == told[6][3] * tile + told[5]


@pytest.mark.parametrize("seed", range(30))
def test_sequences_without_groups_take_their_own_tokens(seed):
    g = np.random.default_rng(800 + seed)
    ns, lens, group, shared, P, width = sp.batch(g)
    taken, _, sh, _ = sp.plan(ns, lens, [-1] * len(ns), shared, 2, 4, 64, P, width, 256, True)
    assert not any(sh) and not any(k[0] for k in taken)
    taken, _, sh, _ = sp.plan(ns, lens, list(range(len(ns))), shared, 2, 4, 64, P, width, 256, True)
    assert not any(sh) and not any(k[0] for k in taken)
