"""The layer's calls without a GPU: what the C entries and the binding refuse.  No kernel runs:
every call returns at an argument check.  A zeroed buffer stands in for the context, of which
these checks read nothing but the number of compute units."""

import ctypes
import os

import pytest
import torch

import fp8_dynamic_quant_amd as wq

pytestmark = pytest.mark.skipif(not os.path.exists(wq.LIB_PATH), reason="libwq.so not built")

NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 6
P = 0x10000  # a 16-byte aligned address that is never read


@pytest.fixture()
def ctx():
    c = ctypes.create_string_buffer(4096)
    ctypes.memmove(ctypes.addressof(c) + 4, ctypes.byref(ctypes.c_int(256)), 4)  # num_cu
    return c


def _norm(ctx, x=P, ldx=512, r=P, ldr=512, gamma=P, M=3, K=512, payload=1, xq=P, xs=P, s=P, lds=512, y=P, ldy=512):
    return wq.lib().wq_add_rms_quant(ctx, x, ldx, r, ldr, gamma, 1e-6, M, K, payload, xq, xs, s, lds, y, ldy, None)


@pytest.mark.parametrize("kw, want", [
    (dict(M=0), 0), (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=-16), SHAPE), (dict(K=24), SHAPE),
    (dict(K=65552, ldx=65552, ldr=65552, lds=65552, ldy=65552), SHAPE), (dict(payload=2, K=64), SHAPE), (dict(payload=3, K=48), SHAPE),
    (dict(payload=0), SHAPE), (dict(payload=6), SHAPE), (dict(payload=4), UNSUPPORTED), (dict(payload=5), UNSUPPORTED),
    (dict(ldx=496), SHAPE), (dict(ldr=496), SHAPE), (dict(lds=496), SHAPE), (dict(ldy=496), SHAPE), (dict(x=None), NULL),
    (dict(gamma=None), NULL), (dict(xq=None), NULL), (dict(xs=None), NULL), (dict(x=P + 2), ALIGN), (dict(r=P + 8), ALIGN),
    (dict(gamma=P + 4), ALIGN), (dict(xq=P + 8), ALIGN), (dict(xs=P + 4), ALIGN), (dict(s=P + 2), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(ldx=516), ALIGN), (dict(ldr=516), ALIGN), (dict(lds=516), ALIGN), (dict(ldy=516), ALIGN),
    (dict(M=0, x=None, xq=None, xs=None, gamma=None), 0)])
def test_norm_refusals(ctx, kw, want):
    assert _norm(ctx, **kw) == want
    assert _norm(None, **kw) == NULL


def _cache(**kw):
    d = wq.KvCacheDesc()
    for k, v in dict(dict(code=1, pages=4, heads=2, page_tokens=16, head_dim=64, k=P, v=P, k_scale=P, v_scale=P, table=P,
                          table_stride=4, max_pages=4), **kw).items():
        setattr(d, k, v)
    return d


def _append(ctx, cache, k=P, ldk=128, v=P, ldv=128, q=P, ldq=512, heads=8, qo=P, ldo=512, angles=P, positions=64, rot=64, T=5, B=2,
            off=P, lens=P):
    return wq.lib().wq_kv_append_rotated(ctx, ctypes.byref(cache), k, ldk, v, ldv, q, ldq, heads, qo, ldo, angles, positions, rot, 0,
                                         T, B, off, lens, None)


def _attend(ctx, cache, q=P, ldq=512, T=5, heads=8, B=2, off=P, lens=P, group=P, shared=P, scale=1.0, out=P, ldo=512, ws=P, n=1 << 40):
    return wq.lib().wq_kv_attention_shared(ctx, ctypes.byref(cache), q, ldq, T, heads, B, off, lens, group, shared, scale, 1, out, ldo,
                                           None, ws, n, None)


@pytest.mark.parametrize("kw, want", [
    (dict(code=0), SHAPE), (dict(pages=0), SHAPE), (dict(heads=0), SHAPE), (dict(page_tokens=24), SHAPE), (dict(page_tokens=272), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(max_pages=0), SHAPE), (dict(table_stride=3), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(k_scale=None), NULL), (dict(v_scale=None), NULL), (dict(table=None), NULL), (dict(k=P + 8), ALIGN), (dict(v=P + 8), ALIGN)])
def test_cache_refusals(ctx, kw, want):
    assert _append(ctx, _cache(**kw)) == want
    assert _attend(ctx, _cache(**kw)) == want


@pytest.mark.parametrize("kw, want", [
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(ldk=120), SHAPE), (dict(ldv=120), SHAPE),
    (dict(rot=0), SHAPE), (dict(rot=8), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(positions=0), SHAPE),
    (dict(positions=1 << 31), SHAPE), (dict(heads=1), SHAPE), (dict(heads=3), SHAPE), (dict(heads=1 << 21), SHAPE), (dict(ldq=504), SHAPE),
    (dict(ldo=504), SHAPE), (dict(q=None), NULL), (dict(qo=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(angles=None), NULL), (dict(off=None), NULL), (dict(lens=None), NULL), (dict(k=P + 2), ALIGN), (dict(v=P + 2), ALIGN),
    (dict(q=P + 8), ALIGN), (dict(qo=P + 8), ALIGN), (dict(angles=P + 4), ALIGN), (dict(ldk=132), ALIGN), (dict(ldv=132), ALIGN),
    (dict(ldq=516), ALIGN), (dict(ldo=516), ALIGN), (dict(q=None, qo=None, T=0), 0)])
def test_append_refusals(ctx, kw, want):
    assert _append(ctx, _cache(), **kw) == want
    assert _append(None, _cache(), **kw) == NULL


@pytest.mark.parametrize("kw, want", [
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), SHAPE), (dict(heads=1), SHAPE), (dict(heads=3), SHAPE), (dict(ldq=504), SHAPE),
    (dict(ldo=504), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(group=None), NULL), (dict(shared=None), NULL), (dict(off=None), NULL), (dict(q=P + 2), ALIGN),
    (dict(out=P + 8), ALIGN), (dict(ldq=516), ALIGN), (dict(ws=P + 4), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=100), WORKSPACE)])
def test_attention_refusals(ctx, kw, want):
    assert _attend(ctx, _cache(), **kw) == want
    assert _attend(None, _cache(), **kw) == NULL


def test_attention_workspace_and_path(ctx):
    L = wq.lib()
    one = _cache(max_pages=8192, table_stride=8192)
    need = lambda T, heads, B: L.wq_kv_attention_shared_workspace_bytes(ctx, ctypes.byref(one), T, heads, B)  # noqa: E731
    path = lambda T, heads, B: L.wq_kv_attention_shared_path(ctx, ctypes.byref(one), T, heads, B)  # noqa: E731
    assert need(0, 8, 1) == 0 and path(0, 8, 1) == 0
    assert need(1, 3, 1) == -SHAPE and path(1, 3, 1) == -SHAPE
    assert L.wq_kv_attention_shared_workspace_bytes(None, ctypes.byref(one), 1, 8, 1) == -NULL
    # two f32 rows and their two numbers for every output row, and a tile for every workgroup
    assert need(64, 8, 64) >= 2 * 64 * 8 * 64 * 4
    assert _attend(ctx, one, T=64, B=64, n=need(64, 8, 64) - 1) == WORKSPACE
    assert path(64, 8, 64) == 16 and path(4096, 32, 16) == L.wq_kv_attention_path(ctx, ctypes.byref(one), 4096, 32, 16) != 16


def test_attention_refuses_work_beyond_52_bits(ctx):
    far = _cache(heads=1024, pages=(1 << 31) - 1, max_pages=(1 << 31) - 1, table_stride=(1 << 31) - 1, page_tokens=256)
    ask = lambda B: wq.lib().wq_kv_attention_shared_workspace_bytes(ctx, ctypes.byref(far), B, 1024, B)  # noqa: E731
    assert ask(1) > 0 and ask(1 << 10) == -SHAPE
    assert _attend(ctx, far, T=1 << 10, B=1 << 10, heads=1024, ldq=65536, ldo=65536) == SHAPE


def test_binding_refusals():
    def bad(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    x = torch.zeros((3, 128), dtype=torch.bfloat16)
    g = torch.ones(128, dtype=torch.bfloat16)
    bad("x must", wq.wq_add_rms_quant, x[None], None, g)
    bad("x must", wq.wq_add_rms_quant, x.float(), None, g)
    bad("x must", wq.wq_add_rms_quant, torch.zeros((128, 3), dtype=torch.bfloat16).t(), None, g)
    bad("residual must", wq.wq_add_rms_quant, x, x[:2], g)
    bad("rms_gamma must", wq.wq_add_rms_quant, x, x, g[:64])
    bad("rms_gamma must", wq.wq_add_rms_quant, x, x, g.float())
    bad("sum_out must", wq.wq_add_rms_quant, x, x, g, sum_out=x.float())
    bad("y must", wq.wq_add_rms_quant, x, x, g, y=x[:, :64])
    bad("x_q must", wq.wq_add_rms_quant, x, x, g, x_q=torch.zeros((3, 1, 128), dtype=torch.int8))
    bad("x_s must", wq.wq_add_rms_quant, x, x, g, x_s=torch.zeros(4))
    c = wq.kv_cache(4, 2, 16, 64, device="cpu")
    off, lens, table = torch.tensor([0, 3]), torch.tensor([3], dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    angles = wq.rotary_angles(8, 32, device="cpu")
    assert angles.shape == (8, 2, 16) and angles.dtype == torch.float32
    bad("angles must", wq.wq_kv_append_rotated, c, k, k, off, lens, table, angles.double())
    bad("angles must", wq.wq_kv_append_rotated, c, k, k, off, lens, table, angles[:, :1])
    bad("k must", wq.wq_kv_append_rotated, c, k[:, :1], k, off, lens, table, angles)
    bad("same number", wq.wq_kv_append_rotated, c, k, k[:2], off, lens, table, angles)
    bad("q must", wq.wq_kv_append_rotated, c, k, k, off, lens, table, angles, q=k[:2])
    bad("q_out", wq.wq_kv_append_rotated, c, k, k, off, lens, table, angles, q_out=k)
    bad("q_out must", wq.wq_kv_append_rotated, c, k, k, off, lens, table, angles, q=k, q_out=k[:2])
    ids = torch.zeros(1, dtype=torch.int32)
    bad("group must", wq.wq_kv_attention_shared, c, k, off, lens, table, ids.long(), ids)
    bad("shared must", wq.wq_kv_attention_shared, c, k, off, lens, table, ids, ids[:0])


def test_angles_are_those_of_64_bits():
    import math

    a = wq.rotary_angles(131072, 64, device="cpu")
    for p, i in ((0, 0), (1, 0), (131071, 0), (131071, 1), (100000, 31)):
        turn = p * 10000.0 ** (-2 * i / 64)
        assert abs(a[p, 0, i].item() - math.cos(turn)) <= 2.0**-24 and abs(a[p, 1, i].item() - math.sin(turn)) <= 2.0**-24
