"""The mapping of workgroups to work in attention behind a shared prefix, restated from the kernels
in whole numbers, and inputs for it."""

import numpy as np

WAVES, TILE, SEQS = 4, 64, 512


def cost_of(rows, D):
    """(tile, units of a step, units of an item besides its steps)."""
    if D < 256 and rows <= 16:
        return 16, 1, 8
    if D == 256 or rows <= 64:
        return 64, 2, 8
    return 128, 3, 12


def plan(ns, lens, group, shared, heads, R, D, P, width, num_runs, causal, least=16):
    """Of one launch: {item: [(run, first step, last step + 1, slot kind, first row of its slots)]},
    the joins as they are told, and the shared steps of each sequence."""
    B = len(ns)
    row0 = np.concatenate(([0], np.cumsum(ns))).astype(int)
    lead, first = [], {}
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

    def own_steps(b):
        seen = min(max(lens[b], 0), width * P)
        return max(max(-(-seen // TILE), 1) - sh[b], 1)

    def units(cost, n):
        return cost[2] + cost[1] * n

    def tiles(cost, rows):
        return -(-rows // cost[0])

    pre = [0]
    for b in range(B):
        rows = ns[b] * R
        v = tiles(cost_of(rows, D), rows) * units(cost_of(rows, D), own_steps(b))
        if lead[b] == b and sh[b] > 0:
            rows = (end[b] - row0[b]) * R
            v += tiles(cost_of(rows, D), rows) * units(cost_of(rows, D), sh[b])
        pre.append(pre[-1] + v)
    total = pre[-1] * heads
    per = max(-(-total // num_runs), least)
    taken, joins = {}, {}

    def at(cost, i0, step):
        return (i0 + cost[2] + step * cost[1]) // per

    for run in range(num_runs):
        u, stop = run * per, min((run + 1) * per, total)
        while u < stop:
            b = max(b for b in range(B) if pre[b] * heads <= u)
            rows, n, base = ns[b] * R, own_steps(b), pre[b] * heads
            cost = cost_of(rows, D)
            own = tiles(cost, rows) * units(cost, n) * heads
            of_group = u - base >= own
            if of_group:
                base += own
                rows, n = (end[b] - row0[b]) * R, sh[b]
                cost = cost_of(rows, D)
            each, t = units(cost, n), tiles(cost, rows)
            item = (u - base) // each
            i0, h, tile = base + item * each, item // t, item % t
            assert h < heads and tile < t and i0 <= u < i0 + each

            def step_at(x):
                return 0 if x <= cost[2] else n if x >= each else -(-(x - cost[2]) // cost[1])

            lo, hi = step_at(u - i0), step_at(stop - i0)
            assert i0 + each > u  # ends
            u = i0 + each
            if lo >= hi:
                continue
            whole = not of_group and sh[b] == 0 and lo == 0 and hi == n
            kind = "out" if whole else "first" if lo == 0 else "run"
            taken.setdefault((of_group, b, h, tile, n, cost[0], rows), []).append((run, lo, hi, kind))
            if lo == 0 and not of_group:
                for r in range(tile * cost[0], min((tile + 1) * cost[0], rows)):
                    told = None
                    if not whole:
                        r0 = at(cost, i0, 0)
                        told = (r0, at(cost, i0, n - 1) - r0 + 1, r - tile * cost[0])
                        if sh[b] > 0:
                            m = lead[b]
                            all_rows, gr = (end[m] - row0[m]) * R, (row0[b] - row0[m]) * R + r
                            k = cost_of(all_rows, D)
                            lr = ns[m] * R
                            kl = cost_of(lr, D)
                            behind = tiles(kl, lr) * units(kl, own_steps(m))
                            i1 = (pre[m] + behind) * heads + (h * tiles(k, all_rows) + gr // k[0]) * units(k, sh[m])
                            r1 = at(k, i1, 0)
                            told += (r1, at(k, i1, sh[m] - 1) - r1 + 1, gr % k[0], (True, m, h, gr // k[0]))
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
