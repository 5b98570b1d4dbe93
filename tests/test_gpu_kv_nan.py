"""Rows of the cache's attention that see a NaN: out and lse are NaN, whatever else they see, in
every form of the attention; a row that sees no token gets zeros and -inf."""

import numpy as np
import pytest
import torch

import kv_forms as kf
from gpu_util import bf16_dev, dev, host, host_bf16_bits, poison
from oracle import numerics as nm
from test_gpu_kv import _limits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_rows_that_see_a_nan(name, D, i8):
    f, c, table, q = kf.inputs(name, D, i8, 3)
    c[2][table[1, 0], 0] = 255                    # keys of a sequence's only page
    c[3][table[1, 0], -1] = 255                   # values of it
    c[2][table[0, :], 0] = 255                    # every page of a sequence
    long = int(np.argmax(f["lens"]))
    c[3][table[long, f["lens"][long] // f["P"] // 2], -1] = 255
    q[int(f["offsets"][long]), 1, D // 2] = 0x7FC0
    q[int(f["offsets"][long]), 2, :] = 0xFFC1
    off, lens, tab = dev(f["offsets"]), dev(np.array(f["lens"], np.int32)), dev(table)
    cache = wq.KvCache(*(dev(x) for x in c))
    assert wq.wq_kv_attention_path(cache, q.shape[0], q.shape[1], tab) == f["path"]
    out, lse = poison(q.shape, torch.bfloat16), poison(q.shape[:2], torch.float32)
    print(f"{name} D={D} i8={i8}", flush=True)
    wq.wq_kv_attention(cache, bf16_dev(q), off, lens, tab, out=out, lse=lse)
    torch.cuda.synchronize()
    want, want_lse, mag, smag = kf.attention(c, q, f["offsets"], f["lens"], table, D**-0.5, True)
    n = int(f["offsets"][-1])
    got, got_lse = nm.bf16_to_f32(host_bf16_bits(out)).astype(np.float64)[:n], host(lse).astype(np.float64)[:n]
    want, want_lse = want[:n], want_lse[:n]
    nan, empty = np.isnan(want_lse), np.isneginf(want_lse)
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(got_lse), nan)
    assert np.array_equal(np.isnan(got).all(-1), nan) and np.array_equal(np.isnan(got).any(-1), nan)
    assert np.array_equal(np.isneginf(got_lse), empty) and not got[empty].any()
    some = ~(nan | empty)
    lim, lim_lse = _limits(np.where(some[..., None], want, 0), np.where(some, want_lse, 0), mag[:n], smag[:n], max(f["lens"]), D)
    assert (np.abs(got - want) <= lim)[some].all() and (np.abs(got_lse - want_lse) <= lim_lse)[some].all()
