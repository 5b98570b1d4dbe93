"""Offsets that the call's contract excludes, in attention behind a shared prefix: they are read as
their running maximum, whatever they hold, and nothing outside the outputs and the workspace is written."""

import ctypes

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from gpu_util import DEV, bf16_dev, dev, host, host_bf16_bits, poison
from oracle import numerics as nm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


@pytest.mark.parametrize("D, B, T", [(64, 5, 40), (128, 13, 30), (128, 200, 150), (256, 9, 30), (64, 512, 300)])
@pytest.mark.parametrize("seed", range(2))
def test_offsets_are_read_as_their_running_maximum(D, B, T, seed):
    H, R, P, width = 2, 4, 32, 9
    g = syn.rng(133, seed, D, B)
    offsets = g.integers(-9, T + 20, B + 1).astype(np.int64)
    offsets[0], offsets[B] = seed * 3, T - 2 * seed
    running = np.maximum.accumulate(np.clip(offsets, 0, T))
    assert (np.diff(offsets) < 0).any()
    c = kf.cache(g, width * 4, H, P, D, False)
    table = np.tile(g.permutation(len(c[0]))[:width], (B, 1)).astype(np.int32)
    lens = g.integers(100, width * P + 1, B).astype(np.int32)
    group = np.cumsum(g.random(B) < 0.3).astype(np.int32)
    shared = g.integers(0, width * P, B).astype(np.int32)
    q = bf16_dev(nm.f64_to_bf16_rn(g.standard_normal((T, H * R, D))))
    cd = wq.KvCache(*(dev(x) for x in c))
    rest = [dev(x) for x in (lens, table, group, shared)]
    d = wq.KvCacheDesc(wq.WQ_KV_E4M3, len(c[0]), H, P, D, *(t.data_ptr() for t in cd), rest[1].data_ptr(), width, width)
    ctx = wq.context(DEV).handle
    need = wq.lib().wq_kv_attention_shared_workspace_bytes(ctx, ctypes.byref(d), T, H * R, B)
    print(f"offsets D={D} B={B} T={T} {offsets[:14].tolist()}", flush=True)
    got = []
    for o in (running, offsets):
        ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
        out, lse, od = poison(q.shape, torch.bfloat16), poison((T, H * R), torch.float32), dev(o)
        assert wq.lib().wq_kv_attention_shared(
            ctx, ctypes.byref(d), q.data_ptr(), H * R * D, T, H * R, B, od.data_ptr(), rest[0].data_ptr(), rest[2].data_ptr(),
            rest[3].data_ptr(), D**-0.5, 1, out.data_ptr(), H * R * D, lse.data_ptr(), ws.data_ptr(), need,
            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert (ws[need:] == 0xFF).all()
        got.append((host_bf16_bits(out), host(lse).view(np.uint32)))
    lo, hi, end = int(running[0]), int(np.clip(offsets[B], 0, T)), int(running[B])
    for a, b in zip(*got):
        assert np.array_equal(a[lo:hi], b[lo:hi])
        for x in (a, b):  # rows of no sequence
            assert (np.concatenate((x[:lo], x[end:])).view(np.uint8) == 0xA5).all()
