"""Calls of attention behind a shared prefix and of the turned append that their contracts allow:
rows inside wider buffers, tables of longer rows, caches beyond 4 GiB."""

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from gpu_util import DEV, bf16_dev, dev, host, host_bf16_bits
from oracle import numerics as nm
from test_gpu_shared import _case, _check

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


@pytest.mark.parametrize("D, i8", [(64, True), (128, False), (256, True)])
@pytest.mark.parametrize("name", ["answers", "drafts", "wide", "chunks"])
def test_rows_in_wider_buffers_and_a_wider_table(name, D, i8):
    # the same numbers lie elsewhere: the same bits come out, and nothing beside them is written
    f, c, table, q = _case(name, D, i8)
    cd, args, out, lse = _check(c, table, q, **f, causal=True)
    n, (T, Hq, _), pad = sum(f["ns"]), q.shape, 24
    qw = torch.full((T, Hq * D + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    qw[:, : Hq * D] = args[0].view(T, -1)
    tw = torch.full((table.shape[0], table.shape[1] + 5), 1 << 30, dtype=torch.int32, device=DEV)
    tw[:, : table.shape[1]] = args[3]
    ow = torch.full((T, Hq * D + 2 * pad), -7.0, dtype=torch.bfloat16, device=DEV)
    view = ow[:, pad : pad + Hq * D].unflatten(1, (Hq, D))
    args[0], args[3] = qw[:, : Hq * D].unflatten(1, (Hq, D)), tw[:, : table.shape[1]]
    _, got_lse = wq.wq_kv_attention_shared(cd, *args, out=view, return_lse=True)
    torch.cuda.synchronize()
    assert np.array_equal(host_bf16_bits(view)[:n], host_bf16_bits(out)[:n])
    assert np.array_equal(host(got_lse)[:n].view(np.uint32), host(lse)[:n].view(np.uint32))
    assert (ow[:, :pad] == -7.0).all() and (ow[:, pad + Hq * D :] == -7.0).all() and (ow[n:] == -7.0).all()


@pytest.mark.parametrize("D, R, ns", [(128, 4, [1, 1, 1]), (128, 8, [20, 9, 30]), (256, 4, [1, 3])])
def test_pages_behind_4_gib(D, R, ns):
    # the last pages of 70,000 (of 64 KiB each for k and v), in attention and in the turned append, against a
    # small cache of the same pages
    P, H, width = 64, 65536 // 64 // D, 8
    pages, B = 70000, len(ns)
    g = syn.rng(135, D, R)
    few = B * width
    small = kf.cache(g, few, H, P, D, False)
    table = np.arange(few).reshape(B, width).astype(np.int32)
    table[1:, :4] = table[0, :4]
    lens = [int(x) for x in g.integers(300, width * P + 1, B)]
    shape_k, shape_v = (pages, H, P, D), (pages, H, D, P)
    big = [torch.empty(s, dtype=torch.uint8, device=DEV) for s in (shape_k, shape_v, (pages, H), (pages, H))]
    for a, b in zip(big, small):
        a[:few] = 0x7F  # E4M3's NaN: what an address of 32 bits would reach
        a[pages - few :] = dev(b)
    big, near = wq.KvCache(*big), wq.KvCache(*(dev(x) for x in small))
    T = sum(ns)
    off = dev(np.concatenate(([0], np.cumsum(ns))).astype(np.int64))
    q, kn, vn = (bf16_dev(nm.f64_to_bf16_rn(g.standard_normal((T, h, D)))) for h in (H * R, H, H))
    rest = [dev(np.array(x, np.int32)) for x in (lens, [0] * B, [4 * P] * B)]
    angles = wq.rotary_angles(width * P, D, device=DEV)
    got = []
    for cache, first in ((near, 0), (big, pages - few)):
        t = dev(table + np.int32(first))
        turned = wq.wq_kv_append_rotated(cache, kn, vn, off, rest[0], t, angles, q=q)
        out, lse = wq.wq_kv_attention_shared(cache, turned, off, rest[0], t, rest[1], rest[2], return_lse=True)
        torch.cuda.synchronize()
        assert torch.isfinite(out.float()).all()
        got.append((turned.view(torch.int16), out.view(torch.int16), lse, *(x[first : first + few].clone() for x in cache)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (big.k[:few] == 0x7F).all() and (big.v[:few] == 0x7F).all()
