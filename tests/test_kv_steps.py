"""The stepping of a wave through its share of a sequence, and of a workgroup's waves through its
items, restated from the attention of 16-row tiles: every step once, every table entry that is
read inside the sequence's, and the same barriers for all four waves, whatever the lengths."""

import numpy as np
import pytest

WAVES, TILE = 4, 64


def steps(lo, hi, stride):
    """(step, step whose page numbers are read for the next round) of one wave, as it goes."""
    taken, reads = [], []
    if lo >= hi:
        return taken, reads
    reads += [lo, min(lo + stride, hi - 1)]
    nstep, step = min(lo + stride, hi - 1), lo
    while step < hi:
        taken.append(step)
        nstep = min(nstep + stride, hi - 1)
        reads.append(nstep)
        step += stride
        assert len(taken) <= hi  # ends
    return taken, reads


@pytest.mark.parametrize("seed", range(50))
def test_waves_share_steps_and_barriers(seed):
    g = np.random.default_rng(600 + seed)
    per = int(g.integers(1, 17))  # token groups of 16 to a page
    width = int(g.integers(1, 60))
    length = int(g.integers(-2, width * per * 16 + 100))
    seen = min(max(length, 0), width * per * 16)
    most = -(-seen // TILE)
    at, barriers = 0, np.zeros(WAVES, int)
    total = max(most, 1)
    while at < total:  # an item in parts, as runs cut it
        n = int(g.integers(1, total - at + 1))
        taken = []
        for wave in range(WAVES):
            mine, reads = steps(at + wave, min(at + n, most), WAVES)
            taken += mine
            for s in reads:
                for group in range(4):
                    tg = 4 * s + group
                    assert 16 * tg >= seen or tg // per < width
            barriers[wave] += 2  # after the sums are in LDS, after they are read
        assert sorted(taken) == list(range(at, min(at + n, most)))
        at += n
    assert (barriers == barriers[0]).all()


def test_pages_by_a_reciprocal():
    # group / per by the upper half of a product, exact up to 2^27 groups (2^31 tokens)
    for per in range(2, 17):
        recip = ((1 << 32) + per - 1) // per
        n = np.concatenate((np.arange(1 << 12), np.random.default_rng(per).integers(0, 1 << 27, 1 << 14), (1 << 27) - 1 - np.arange(1 << 10)))
        n = np.concatenate((n, n // per * per)).astype(np.uint64)
        assert np.array_equal(n * np.uint64(recip) >> np.uint64(32), n // np.uint64(per))
