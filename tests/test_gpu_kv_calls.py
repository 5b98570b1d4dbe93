"""How the cache's attention is called, in every form: workspaces that hold anything and no byte
more than asked for, the context's own, captured graphs with eager calls between their replays, two
streams at once; the same bytes each time."""

import ctypes

import numpy as np
import pytest
import torch

import kv_forms as kf
from gpu_util import bf16_dev, dev, host, host_bf16_bits, poison
from oracle import numerics as nm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


def _set(name, D, i8, seed):
    f, c, table, q = kf.inputs(name, D, i8, seed)
    return wq.KvCache(*(dev(x) for x in c)), bf16_dev(q), dev(f["offsets"]), dev(np.array(f["lens"], np.int32)), dev(table)


def _bits(out, lse):
    return host_bf16_bits(out), host(lse).view(np.uint32)


def _same(a, b):
    return all(np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_workspaces(name, D, i8):
    cache, q, off, lens, table = _set(name, D, i8, 20)
    n = int(host(off)[-1])
    T, heads, _ = q.shape
    want = [x[:n] for x in _bits(*wq.wq_kv_attention(cache, q, off, lens, table, return_lse=True))]
    pages, H, P, _ = cache.k.shape
    d = wq.KvCacheDesc(wq.WQ_KV_INT8 if i8 else wq.WQ_KV_E4M3, pages, H, P, D, *(t.data_ptr() for t in cache), table.data_ptr(),
                       table.shape[1], table.shape[1])
    ctx = wq.context(q.device).handle
    need = wq.lib().wq_kv_attention_workspace_bytes(ctx, ctypes.byref(d), T, heads, len(lens))
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    print(f"{name} D={D} i8={i8} workspace {need}", flush=True)
    for at, size in ((ws.data_ptr(), need), (None, 0)):
        out, lse = poison(q.shape, torch.bfloat16), poison((T, heads), torch.float32)
        args = (q.data_ptr(), heads * D, T, heads, len(lens), off.data_ptr(), lens.data_ptr(), D**-0.5, 1, out.data_ptr(), heads * D,
                lse.data_ptr(), at, size, torch.cuda.current_stream().cuda_stream)
        assert wq.lib().wq_kv_attention(ctx, ctypes.byref(d), *args) == 0
        torch.cuda.synchronize()
        assert _same([x[:n] for x in _bits(out, lse)], want)
    assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("name, D, i8", [(n, D, i8) for n in sorted(kf.FORMS) for D, i8 in ((64, True), (128, False), (256, True))])
def test_graphs_with_eager_calls_between(name, D, i8):
    cache, q, off, lens, table = _set(name, D, i8, 21)
    n = int(host(off)[-1])
    wq.wq_kv_attention(cache, q, off, lens, table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = wq.wq_kv_attention(cache, q, off, lens, table, return_lse=True)
    print(f"{name} D={D} i8={i8}", flush=True)
    g = np.random.default_rng(1)
    for i in range(4):
        q.copy_(bf16_dev(nm.f64_to_bf16_rn(g.standard_normal(q.shape))))
        if i:  # shorter sequences, other pages: the plan follows them
            lens.copy_((lens - int(g.integers(0, 20))).clamp(min=0))
            table.copy_(table.flip(1))
        graph.replay()
        eager = wq.wq_kv_attention(cache, q, off, lens, table, return_lse=True)
        torch.cuda.synchronize()
        assert _same([x[:n] for x in _bits(out, lse)], [x[:n] for x in _bits(*eager)])


@pytest.mark.parametrize("name, D", [(n, D) for n in sorted(kf.FORMS) for D in (64, 256)])
def test_two_streams_at_once(name, D):
    sets = [_set(name, D, bool(i), 22 + i) for i in range(2)]
    n = int(host(sets[0][2])[-1])
    want = [[x[:n] for x in _bits(*wq.wq_kv_attention(*s, return_lse=True))] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    print(f"{name} D={D}", flush=True)
    got = []
    for _ in range(6):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(wq.wq_kv_attention(*s, return_lse=True))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert _same([x[:n] for x in _bits(*o)], want[i % 2])
