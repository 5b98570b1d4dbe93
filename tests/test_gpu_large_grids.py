"""Calls whose workgroups one axis of a launch does not count (2^32 threads): the same bytes as the
same rows in smaller calls."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq

DEV = "cuda"


def _rows(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).bfloat16()


@pytest.mark.parametrize("T", [(1 << 26) + 5, (1 << 28) + 3])
def test_blocks_of_many_tokens(T):
    # 2^22 + 1 and 2^24 + 1 workgroups; tokens repeat with an odd period
    print(f"T={T}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(1)
    period = 524287
    one = _rows(gen, period, 1, 32) * torch.exp(_rows(gen, period, 1, 1).float()).bfloat16()
    q1, _, s1 = wq.wq_group_quant_mxfp4(one)
    y1 = wq.wq_group_dequant_mxfp4(q1, s1)
    x = torch.empty((T, 1, 32), dtype=torch.bfloat16, device=DEV)
    whole = T // period * period
    x[:whole].view(-1, period, 1, 32)[:] = one
    x[whole:] = one[: T - whole]
    q, _, s = wq.wq_group_quant_mxfp4(x)
    del x
    s, y = s.view(-1), wq.wq_group_dequant_mxfp4(q, s)
    assert not s[T:].any()
    for got, want in ((q, q1), (s[:T], s1.view(-1)[:period]), (y.view(torch.int16), y1.view(torch.int16))):
        for part in got[:whole].view(-1, *want.shape).split(64):
            assert torch.equal(part, want.expand_as(part))
        assert torch.equal(got[whole:], want[: T - whole])


def _cache(gen, pages, H, P, D):
    c = wq.kv_cache(pages, H, P, D, dtype=torch.int8)
    for t in c[:2]:
        for part in t.split(max(1, (1 << 30) // (H * P * D))):
            part.copy_(torch.randint(-127, 128, part.shape, generator=gen, device=DEV, dtype=torch.int8))
    for t in c[2:]:
        t.fill_(120)
    return c


@pytest.mark.parametrize("by_pages", [False, True])
def test_rows_appended_to_many_sequences(by_pages):
    # a slot a row, and slots by pages: of each more than 2^22
    B = 1 << 22 if not by_pages else 1 << 21
    n = 1 if not by_pages else 6
    print(f"B={B} n={n}", flush=True)
    B += 9
    gen = torch.Generator(device=DEV).manual_seed(2)
    k, v = (_rows(gen, B * n, 1, 64) for _ in range(2))
    off = torch.arange(B + 1, device=DEV) * n
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    table = torch.arange(B, dtype=torch.int32, device=DEV).flip(0)[:, None]
    c = wq.kv_cache(B, 1, 16, 64)
    wq.wq_kv_append(c, k, v, off, lens, table)
    d = wq.kv_cache(B, 1, 16, 64)
    for b in range(0, B, 1 << 20):
        to = min(B, b + (1 << 20))
        wq.wq_kv_append(d, k[b * n : to * n], v[b * n : to * n], off[b : to + 1] - b * n, lens[b:to], table[b:to])
    for x, y in zip(c, d):
        assert x.any() and torch.equal(x, y)


@pytest.mark.parametrize("B, H, path", [((1 << 20) + 3, 8, 1), (127, 65535, 2)])
def test_attention_of_many_sequences_and_heads(B, H, path):
    # whole row tiles of more than 2^22 (sequence, head) pairs; as many items, several to a workgroup
    print(f"B={B} H={H}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(3)
    c = _cache(gen, B, H, 16, 64)
    table = torch.randperm(B, generator=gen, device=DEV).int()[:, None]
    lens = torch.randint(0, 17, (B,), generator=gen, device=DEV).int()
    off = torch.arange(B + 1, device=DEV)
    q = _rows(gen, B, H, 64)
    assert wq.wq_kv_attention_path(c, B, H, table) == path
    out, lse = wq.wq_kv_attention(c, q, off, lens, table, return_lse=True)
    part = 1 << 18 if path == 1 else 32
    for b in range(0, B, part):
        n = min(part, B - b)
        if path == 1 and n <= 4096:  # the last few would take another form
            b, n = B - part, part
        assert wq.wq_kv_attention_path(c, n, H, table[b : b + n]) == path
        o, l = wq.wq_kv_attention(c, q[b : b + n], off[: n + 1], lens[b : b + n], table[b : b + n], return_lse=True)
        assert torch.equal(out[b : b + n].view(torch.int16), o.view(torch.int16)) and torch.equal(lse[b : b + n], l)
    assert torch.isfinite(out[lens > 0]).all() and not out[lens == 0].any()
