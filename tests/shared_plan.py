"""The mapping of workgroups to work in attention behind a shared prefix, restated from the kernels
in whole numbers, and inputs for it."""

import numpy as np

TILE, SEQS, WAVES = 64, 512, 8
NARROW, WIDE = 0, 1
FIXED = (4, 6)  # units that an item counts besides its steps


def kind_of(rows, D):
    """(kind, rows of a tile)."""
    if D < 256 and rows <= 16:
        return NARROW, 16
    return WIDE, 128 if D == 256 else 256


def plan(ns, lens, group, shared, heads, R, D, P, width, workgroups, causal, least=(5, 2)):
    """Of one launch: {item: [(run, first step, last step + 1, slot kind)]}, the joins as they are
    told, the shared steps of each sequence and the one whose table it takes them from."""
    B = len(ns)
    row0 = np.concatenate(([0], np.cumsum(ns))).astype(int)
    lead = []
    for b in range(B):
        begins = b > 0 and (group[b] < 0 or group[b] != group[b - 1])
        lead.append(b if begins or b == 0 else lead[-1])
    steps, end, many, holder = {}, {}, {}, {}
    for b in range(B):
        if ns[b] > 0:
            own = max(min(shared[b], min(lens[b] - (ns[b] if causal else 0), width * P)), 0)
            m = lead[b]
            steps[m] = min(steps.get(m, 1 << 31), own // P * P // TILE)
            end[m] = max(end.get(m, 0), row0[b + 1])
            many[m] = many.get(m, 0) + 1
            holder.setdefault(m, b)
    sh = [steps[lead[b]] if many.get(lead[b], 0) > 1 else 0 for b in range(B)]

    def items(rows, n):
        """(kind, rows of a tile, tiles, steps, units of an item)."""
        kind, tile = kind_of(rows, D)
        return kind, tile, -(-rows // tile), n, n + FIXED[kind]

    def own_items(b):
        seen = min(max(lens[b], 0), width * P)
        return items(ns[b] * R, max(max(-(-seen // TILE), 1) - sh[b], 1))

    def group_items(m):
        return items((end[m] - row0[m]) * R, sh[m])

    pre = [[0], [0]]
    for b in range(B):
        v = [0, 0]
        for k in [own_items(b)] + ([group_items(b)] if lead[b] == b and sh[b] > 0 else []):
            v[k[0]] += k[2] * k[4]
        for x in (0, 1):
            pre[x].append(pre[x][-1] + v[x])
    taken, joins = {}, {}
    assert workgroups > 1  # some for either kind
    units = [pre[x][-1] * heads for x in (0, 1)]
    share = workgroups * units[WIDE] // (units[WIDE] + -(-units[NARROW] * 5 // (4 * WAVES)) + 1)
    wide = workgroups if units[NARROW] == 0 else min(max(share, 1), workgroups - 1)
    per_wide = max(-(-units[WIDE] // wide), least[WIDE])
    wide = -(-units[WIDE] // per_wide)  # workgroups that take wide runs; the others' waves take narrow ones
    narrow = (workgroups - min(wide, workgroups - 1)) * WAVES
    per = (max(-(-units[NARROW] // narrow), least[NARROW]), per_wide)
    runs = (narrow, wide)
    assert units[NARROW] == 0 or wide < workgroups

    def told_of(k, i0, row):
        first = i0 + FIXED[k[0]]
        run = first // per[k[0]]
        return run, (first + k[3] - 1) // per[k[0]] - run + 1, row % k[1]

    for axis in (NARROW, WIDE):
        total = pre[axis][-1] * heads
        for run in range(runs[axis]):
            u, stop = run * per[axis], min((run + 1) * per[axis], total)
            while u < stop:
                b = max(b for b in range(B) if pre[axis][b] * heads <= u)
                k, base = own_items(b), pre[axis][b] * heads
                own = k[2] * k[4] * heads if k[0] == axis else 0
                of_group = u - base >= own
                if of_group:
                    base += own
                    k = group_items(b)
                kind, size, tiles, n, each = k
                assert kind == axis
                item = (u - base) // each
                i0, h, tile = base + item * each, item // tiles, item % tiles
                assert h < heads and tile < tiles and i0 <= u < i0 + each

                def step_at(x):
                    return 0 if x <= FIXED[kind] else min(x - FIXED[kind], n)

                lo, hi = step_at(u - i0), step_at(min(stop - i0, each))
                u = i0 + each  # ends: beyond where it was
                if lo >= hi:
                    continue
                whole = not of_group and sh[b] == 0 and lo == 0 and hi == n
                rows = (end[b] - row0[b]) * R if of_group else ns[b] * R
                taken.setdefault((of_group, b, h, tile), []).append((run, lo, hi, "out" if whole else "first" if lo == 0 else "run", kind, n))
                if lo == 0 and not of_group:
                    for r in range(tile * size, min((tile + 1) * size, rows)):
                        told = None
                        if not whole:
                            told = told_of(k, i0, r)
                            if sh[b] > 0:
                                m = lead[b]
                                gr, g, first = (row0[b] - row0[m]) * R + r, group_items(m), own_items(m)
                                behind = first[2] * first[4] if first[0] == g[0] else 0
                                i1 = (pre[g[0]][m] + behind) * heads + (h * g[2] + gr // g[1]) * g[4]
                                told += told_of(g, i1, gr) + ((True, m, h, gr // g[1]),)
                        joins[(b, h, r)] = told
    return taken, joins, sh, [holder.get(lead[b], b) for b in range(B)]


def batch(g, *, most=12, long=2000):
    """Random sequences, some of them without rows, in groups with what they share."""
    B = int(g.integers(1, most))
    ns = (g.choice([1, 1, 1, 2, 5, 20, 70], B) * (g.random(B) < 0.85)).tolist()
    ns[int(g.integers(B))] = int(g.integers(1, 5))
    group = np.cumsum(g.random(B) < 0.3).tolist()
    if g.random() < 0.3:
        group[int(g.integers(B))] = -1
    P = int(g.choice([16, 32, 48, 64, 128, 256]))
    width = int(g.integers(1, max(2, long // P)))
    lens = [int(x) for x in g.integers(-3, width * P + 100, B)]
    shared = [int(x) for x in g.integers(-5, width * P + 70, B)]
    return ns, lens, group, shared, P, width
