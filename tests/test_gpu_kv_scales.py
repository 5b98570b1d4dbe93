"""The cache's attention with page scales far apart and with score scales at either end of what a
float holds, in every form: keys' and values' bytes over forty powers of two between pages, pages
of byte 0 and 254, score scales from 2^-140 to 2^126."""

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from gpu_util import bf16_dev, dev, host, host_bf16_bits, poison
from oracle import numerics as nm
from test_gpu_kv import _limits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


def _check(name, f, c, table, q, scale, causal=True):
    D = q.shape[2]
    off, lens, tab = dev(f["offsets"]), dev(np.array(f["lens"], np.int32)), dev(table)
    cache = wq.KvCache(*(dev(x) for x in c))
    assert wq.wq_kv_attention_path(cache, q.shape[0], q.shape[1], tab) == f["path"]
    out, lse = poison(q.shape, torch.bfloat16), poison(q.shape[:2], torch.float32)
    print(f"{name} D={D} {c[0].dtype} scale={scale}", flush=True)
    wq.wq_kv_attention(cache, bf16_dev(q), off, lens, tab, out=out, lse=lse, scale=scale, causal=causal)
    torch.cuda.synchronize()
    want, want_lse, mag, smag = kf.attention(c, q, f["offsets"], f["lens"], table, scale, causal)
    n = int(f["offsets"][-1])
    got, got_lse = nm.bf16_to_f32(host_bf16_bits(out)).astype(np.float64)[:n], host(lse).astype(np.float64)[:n]
    empty = np.isneginf(want_lse[:n])
    lim, lim_lse = _limits(want, np.where(np.isneginf(want_lse), 0, want_lse), mag, smag, max(f["lens"]), D)
    assert np.array_equal(np.isneginf(got_lse), empty) and not got[empty].any()
    bad = np.argwhere(~(np.abs(got - want[:n]) <= lim[:n]))
    assert not len(bad), (len(bad), bad[:3].tolist(), got[tuple(bad[0])], want[tuple(bad[0])], lim[tuple(bad[0])])
    assert (np.abs(got_lse - want_lse[:n]) <= lim_lse[:n])[~empty].all()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_page_scales_over_forty_powers_of_two(name, D, i8):
    f, c, table, q = kf.inputs(name, D, i8, 4)
    g = syn.rng(81, D, int(i8))
    top = 122 if i8 else 129  # scores stay as large as they are in the other tests
    c[2] = g.integers(top - 41, top, c[2].shape).astype(np.uint8)
    c[3] = g.integers(100, 141, c[3].shape).astype(np.uint8)
    for causal in (True, False):
        _check(name, f, c, table, q, -(D**-0.5), causal)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_score_scales_that_a_page_takes_out_of_range(name, D, i8):
    """Every other page's keys are zeros with byte 0 or 254: scores of zero whatever the product
    of the two scales, also for the tokens of those pages that a row does not see."""
    f, c, table, q = kf.inputs(name, D, i8, 5)
    for byte, scale in ((0, 2.0**-30), (0, -(2.0**-140)), (254, 2.0**-20)):
        c[0][::2], c[2][::2] = 0, byte
        _check(name, f, c, table, q, scale)
    c[0][:], c[2][:] = 0, 254
    c[2][::3] = 0
    for scale in (4.0, 2.0**126):
        _check(name, f, c, table, q, scale)
