"""The arithmetic that cuts attention behind a shared prefix into runs, built for the CPU from the header
that the kernels take it from, against its restatement in shared_plan: the same runs, steps and parts
for every item, and parts that lie apart and inside the workspace."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import shared_plan as sp

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_dynamic_quant_amd", "csrc")

SHIM = """
#include "wq_kv_plan.h"
using namespace wq;
static Kind kind(int D, uint32_t rows, uint32_t steps) { return D == 256 ? kind_of<256>(rows, steps) : kind_of<64>(rows, steps); }
extern "C" {
void item(int D, uint32_t rows, uint32_t steps, uint32_t* out) {
  const Kind k = kind(D, rows, steps);
  out[0] = k.kind, out[1] = k.tile, out[2] = k.tiles, out[3] = k.units;
}
void axes(uint32_t narrow, uint32_t wide, uint32_t all, uint32_t* out) {
  const SharePlan p = cut_axes(narrow, wide, all);
  for (int i = 0; i < 2; ++i) out[2 * i] = p.axis[i].per, out[2 * i + 1] = p.axis[i].runs;
}
uint32_t step(int D, uint32_t rows, uint32_t steps, uint32_t x) { return step_at(kind(D, rows, steps), x); }
void parts(int D, uint32_t rows, uint32_t steps, uint32_t narrow, uint32_t wide, uint32_t all, uint32_t i0, uint32_t row, uint32_t* out) {
  const Parts t = parts_of(kind(D, rows, steps), cut_axes(narrow, wide, all), i0, row);
  out[0] = t.run, out[1] = t.count, out[2] = t.at;
}
int64_t first(int64_t keys, int64_t key, int of_group) { return first_slot(keys, key, of_group); }
int64_t later(int D, int64_t keys, uint32_t all, int k, uint32_t run, uint32_t row) {
  return D == 256 ? run_slot<256>(keys, all, k, run, row) : run_slot<64>(keys, all, k, run, row);
}
int64_t slots(int64_t keys, uint32_t all, int D) { return share_slots(keys, all, D); }
int sequences() { return kShareSeqs; }
}
"""


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("plan")
    (at / "shim.cpp").write_text(SHIM)
    # what a device compiler knows by itself means nothing here
    subprocess.run([gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-D__host__=", "-D__device__=", "-D__forceinline__=inline", "-I", CSRC,
                    str(at / "shim.cpp"), "-o", str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(str(at / "shim.so"))
    for name in ("first", "later", "slots"):
        getattr(lib, name).restype = ctypes.c_int64
    lib.first.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    lib.later.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint32]
    lib.slots.argtypes = [ctypes.c_int64, ctypes.c_uint32, ctypes.c_int]
    return lib


def _call(fn, *args, n):
    out = (ctypes.c_uint32 * n)()
    fn(*args, out)
    return tuple(out)


def test_constants(code):
    assert code.sequences() == sp.SEQS


@pytest.mark.parametrize("seed", range(60))
def test_runs_are_the_restated_ones(code, seed):
    g = np.random.default_rng(740 + seed)
    ns, lens, group, shared, P, width = sp.batch(g)
    D, heads, R = int(g.choice([64, 256])), int(g.integers(1, 6)), int(g.choice([1, 4, 5, 16]))
    causal, all_ = bool(g.random() < 0.7), int(g.choice([2, 3, 7, 64, 256]))
    taken, joins, sh, _ = sp.plan(ns, lens, group, shared, heads, R, D, P, width, all_, causal)
    B = len(ns)
    row0 = np.concatenate(([0], np.cumsum(ns))).astype(int)
    # the items in order: (of a group, sequence), rows, steps
    items = []
    for b in range(B):
        steps = max(max(-(-min(max(lens[b], 0), width * P) // sp.TILE), 1) - sh[b], 1)
        items.append((False, b, ns[b] * R, steps))
        if (True, b, 0, 0) in taken:
            end = max(row0[x + 1] for x in range(b, B) if ns[x] and all(group[y] == group[b] for y in range(b, x + 1)))
            items.append((True, b, int(end - row0[b]) * R, sh[b]))
    units, starts, kinds = [0, 0], {}, {}
    for of_group, b, rows, steps in items:
        kinds[of_group, b] = k = _call(code.item, D, rows, steps, n=4)
        starts[of_group, b] = units[k[0]] * heads
        units[k[0]] += k[2] * k[3]
    total = [u * heads for u in units]
    per = _call(code.axes, total[0], total[1], all_, n=4)
    keys, used = int(row0[-1]) * R * heads, set()
    seen = set()
    for of_group, b, rows, steps in items:
        kind, tile, tiles, each = kinds[of_group, b]
        for h in range(heads):
            for t in range(tiles):
                seen.add((of_group, b, h, t))
                mine, i0 = taken[of_group, b, h, t], starts[of_group, b] + (h * tiles + t) * each
                told = _call(code.parts, D, rows, steps, total[0], total[1], all_, i0, t * tile, n=3)
                assert told == (mine[0][0], len(mine), kind << 15)
                for run, lo, hi, how, axis, n in mine:
                    u = max(run * per[2 * kind], i0)
                    assert axis == kind and run < per[2 * kind + 1] and n == steps
                    assert code.step(D, rows, steps, u - i0) == lo
                    assert code.step(D, rows, steps, min((run + 1) * per[2 * kind] - i0, each)) == hi
                    for r in range(min(tile, rows - t * tile)):
                        if how == "out":
                            continue
                        if lo == 0:
                            token, head = row0[b] + (t * tile + r) // R, h * R + (t * tile + r) % R
                            at = code.first(keys, int(token) * heads * R + head, of_group)
                        else:
                            at = code.later(D, keys, all_, kind, run, r)
                        assert at not in used and 0 <= at < code.slots(keys, all_, D)
                        used.add(at)
    assert seen == set(taken)


def test_axes_at_the_ends(code):
    # no units of a kind, one workgroup's worth, sums near 2^31
    for narrow, wide in ((0, 0), (0, 7), (7, 0), (1, 1), ((1 << 31) - 1, 5), (5, (1 << 31) - 1), (1 << 30, 1 << 30)):
        for all_ in (2, 3, 256):
            n_per, n_runs, w_per, w_runs = _call(code.axes, narrow, wide, all_, n=4)
            assert n_per * n_runs >= narrow and w_per * w_runs >= wide and (n_runs == 0) == (narrow == 0) and (w_runs == 0) == (wide == 0)
            assert w_runs <= all_ - (narrow > 0) and n_runs <= (all_ - w_runs) * sp.WAVES and n_per >= 5 and w_per >= 2
