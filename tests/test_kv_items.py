"""Items that are not cut, in fewer runs than items (restated from the kernels): each once and whole."""

import numpy as np
import pytest

from test_mx4_kv_calls import attention_runs


@pytest.mark.parametrize("seed", range(40))
def test_a_run_takes_several_items(seed):
    g = np.random.default_rng(500 + seed)
    B, heads, R, krows = int(g.integers(1, 10)), int(g.integers(1, 6)), int(g.choice([1, 4, 5, 16])), int(g.choice([16, 64]))
    ns = (g.integers(0, 20, B) * (g.random(B) < 0.8)).tolist()
    ns[0] += 1
    tiles = sum(-(-n * R // krows) for n in ns)
    done, joins = attention_runs(ns, g.integers(-3, 600, B).tolist(), heads, R, krows, int(g.integers(1, tiles * heads + 1)), 1, 8, False, 512)
    assert len(done) == tiles * heads and not joins
    assert all(len(parts) == 1 and parts[0][0] == 0 for parts in done.values())
