"""Which kernel the 4-bit products and the cache's attention take for which sizes: the host calls
that say so, on a context of 256 compute units (a buffer that holds nothing but their number)."""

import ctypes
import os

import pytest
import torch

import fp8_dynamic_quant_amd as wq

pytestmark = pytest.mark.skipif(not os.path.exists(wq.LIB_PATH), reason="libwq.so not built")

NULL, SHAPE = 1, 2


@pytest.fixture()
def ctx():
    c = ctypes.create_string_buffer(4096)
    ctypes.memmove(ctypes.addressof(c) + 4, ctypes.byref(ctypes.c_int(256)), 4)  # its second int
    return c


@pytest.mark.parametrize("M, N, K, G, want", [
    (0, 64, 128, 1, 0), (1, 1024, 4096, 1, 1), (16, 8176, 128, 1, 1), (16, 8192, 128, 1, 2), (1, 1040, 128, 8, 2),
    (1, 16320, 128, 1, 2), (1, 16336, 128, 1, 3), (17, 16, 128, 1, 3), (64, 1024, 4096, 8, 3), (1000, 2064, 1152, 1, 4),
    (8192, 32768, 1024, 1, 5), (2048, 4096, 4096, 1, 5),
    (-1, 64, 128, 1, -SHAPE), (1, 24, 128, 1, -SHAPE), (1, 64, 192, 1, -SHAPE), (1, 64, 128, 0, -SHAPE), (1, 64, 128, 65536, -SHAPE),
    (1, 64, 131200, 1, -SHAPE), (1, 0, 128, 1, -SHAPE), ((1 << 30) + 1, 64, 128, 1, -SHAPE)])
def test_products(ctx, M, N, K, G, want):
    assert wq.lib().wq_mx4_path(ctx, M, N, K, G) == want
    assert wq.lib().wq_mx4_path(None, M, N, K, G) == -NULL


def _path(ctx, T, q_heads, B, **kw):
    d = wq.KvCacheDesc()
    for k, v in dict(dict(code=1, pages=4, heads=8, page_tokens=16, head_dim=128, max_pages=64, table_stride=64), **kw).items():
        setattr(d, k, v)
    return wq.lib().wq_kv_attention_path(ctx, ctypes.byref(d), T, q_heads, B)


@pytest.mark.parametrize("T, q_heads, B, kw, want", [
    (0, 32, 1, {}, 0), (1, 32, 0, {}, 0),
    (1, 32, 1, {}, 2), (64, 32, 64, dict(page_tokens=64, max_pages=128), 4), (1, 32, 1, dict(max_pages=8192), 4 + 8),
    (40, 32, 2, dict(max_pages=32), 3), (40, 32, 2, {}, 5), (1, 32, 1, dict(head_dim=256), 5),
    (4, 16, 1, dict(heads=1, head_dim=256, max_pages=8192), 5 + 8),
    (1023, 32, 3, {}, 5), (1024, 32, 3, {}, 1), (511, 32, 3, dict(head_dim=256), 5), (512, 32, 3, dict(head_dim=256), 1),
    (1024, 32, 1024, {}, 2), (1024, 32, 1024, dict(max_pages=256), 4), (1024, 32, 1024, dict(max_pages=32), 1),
    (1024, 32, 1024, dict(head_dim=256), 1), (256, 128, 256, {}, 2), (4096, 32, 4097, {}, 1), (1025, 32, 1024, dict(max_pages=256), 1), (4096, 32, 240, {}, 1),
    (4000, 32, 2, {}, 1), (1, 12, 1, {}, -SHAPE), (-1, 32, 1, {}, -SHAPE), (1, 32, 1, dict(head_dim=96), -SHAPE)])
def test_attention(ctx, T, q_heads, B, kw, want):
    assert _path(ctx, T, q_heads, B, **kw) == want
    assert _path(None, T, q_heads, B, **kw) == -NULL


def test_products_of_more_tiles_than_a_launch_counts(ctx):
    d = wq.MatmulDesc()
    for k, v in dict(payload=4, epilogue=1, M=32769, N=16, K=128, batch=65535, a=1 << 16, lda=64, a_batch_stride=1 << 21,
                     a_scale=1 << 16, a_scale_tokens=32772, b=1 << 16, b_batch_stride=1024, b_scale=1 << 16, y=1 << 16, ldy=16,
                     y_batch_stride=1 << 20).items():
        setattr(d, k, v)
    assert wq.lib().wq_quant_matmul(ctx, ctypes.byref(d), None) == SHAPE


@pytest.mark.parametrize("kw", [dict(mx=True), dict(a_scale_tokens=8), dict(n=32)])
def test_arguments_that_contradict_the_operands(kw):
    a, sa = torch.zeros((3, 1, 64), dtype=torch.uint8), torch.zeros((1, 1, 4), dtype=torch.int32)
    w, sw = torch.zeros((1, 16, 64), dtype=torch.uint8), torch.zeros((1, 1, 16), dtype=torch.int32)
    with pytest.raises(ValueError):
        wq.wq_quant_matmul(a, sa, w, sw, fp8_groups=1, mx4=True, **kw)
    for good in ({}, dict(a_scale_tokens=4), dict(n=16)):  # accepted, up to the device
        with pytest.raises(RuntimeError, match="GPU only"):
            wq.wq_quant_matmul(a, sa, w, sw, fp8_groups=1, mx4=True, **good)
