"""Every form of the cache's attention (whole row tiles, 16-row and 64-row tiles as items, as equal
runs and as parts of few items) against the definition, each call asked first which form it takes."""

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


def _check(name, f, c, table, q, *, causal=True, spoil=None, qpad=0, opad=0):
    T, heads, D = q.shape
    n = int(f["offsets"][-1])
    want, want_lse, mag, smag = kf.attention(c, q, f["offsets"], f["lens"], table, D**-0.5, causal)
    if spoil:
        spoil(c)
    cache = wq.KvCache(*(dev(x) for x in c))
    off, lens, tab = dev(f["offsets"]), dev(np.array(f["lens"], np.int32)), dev(table)
    assert wq.wq_kv_attention_path(cache, T, heads, tab) == f["path"]
    wide = torch.full((T, heads * D + qpad), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, : heads * D] = bf16_dev(q).view(T, heads * D)
    out, lse = poison((T, heads * D + opad), torch.bfloat16), poison((T, heads), torch.float32)
    before, before_lse = host_bf16_bits(out), host(lse)
    print(f"{name} D={D} {c[0].dtype} P={f['P']} causal={causal}", flush=True)
    wq.wq_kv_attention(cache, wide[:, : heads * D].unflatten(1, (heads, D)), off, lens, tab, causal=causal,
                       out=out[:, : heads * D].unflatten(1, (heads, D)), lse=lse)
    torch.cuda.synchronize()
    bits, got_lse = host_bf16_bits(out), host(lse)
    assert np.array_equal(bits[n:], before[n:]) and np.array_equal(bits[:, heads * D :], before[:, heads * D :])
    assert np.array_equal(got_lse[n:], before_lse[n:])
    got = nm.bf16_to_f32(bits[:n, : heads * D]).astype(np.float64).reshape(n, heads, D)
    empty = np.isneginf(want_lse[:n])
    lim, lim_lse = _limits(want, np.where(np.isneginf(want_lse), 0, want_lse), mag, smag, max(f["lens"]), D)
    assert np.array_equal(np.isneginf(got_lse[:n]), empty) and not got[empty].any()
    bad = np.argwhere(~(np.abs(got - want[:n]) <= lim[:n]))
    assert not len(bad), (len(bad), bad[:3].tolist(), got[tuple(bad[0])], want[tuple(bad[0])], lim[tuple(bad[0])])
    assert (np.abs(got_lse[:n] - want_lse[:n]) <= lim_lse[:n])[~empty].all()


def _behind(f, table, i8):
    """What may lie behind a sequence's length: any codes, and pages marked NaN."""
    def spoil(c):
        used = np.zeros(len(c[0]), bool)
        for b, length in enumerate(f["lens"]):
            for i, page in enumerate(table[b]):
                if not 0 <= page < len(used):
                    continue
                keep = min(max(length - i * f["P"], 0), f["P"])
                used[page] = keep > 0
                c[0][page, :, keep:], c[1][page, :, :, keep:] = (-128, 127) if i8 else (0x7F, 0xFF)
        c[2][~used], c[3][~used] = 255, 255

    return spoil


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_every_form(name, D, i8, causal):
    f, c, table, q = kf.inputs(name, D, i8, 6, extra=3)
    _check(name, f, c, table, q, causal=causal, spoil=_behind(f, table, i8), qpad=24, opad=40)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", sorted(kf.FORMS))
def test_every_form_without_some_pages(name, D, i8):
    f, c, table, q = kf.inputs(name, D, i8, 7)
    long = int(np.argmax(f["lens"]))
    table[long, 1], table[long, f["lens"][long] // f["P"]] = -1, len(c[0])
    table[1] = 1 << 30
    table[0, 0] = -(1 << 31)
    for causal in (True, False):
        _check(name, f, c, table, q, causal=causal)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P, width", [(16, 24), (48, 8), (80, 5), (128, 3), (256, 2)])
def test_whole_row_tiles_over_every_page(P, width, D, i8):
    f, c, table, q = kf.inputs("rows", D, i8, 8, P=P, width=width)
    _check("rows", f, c, table, q, spoil=_behind(f, table, i8))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_whole_row_tiles_of_prompts_behind_a_cache(D, i8):
    # more rows than tokens, rows that see nothing, one row, odd heads; several tiles of each
    f, c, table, q = kf.inputs("rows", D, i8, 9, ns=[300, 1, 257, 20], lens=[2300, 700, 257, 9], H=5, R=12, P=64, width=36)
    for causal in (True, False):
        _check("rows", f, c, table, q, causal=causal)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("name, D, B, R, width", [("items16", 64, 1030, 12, 9), ("runs16", 128, 600, 16, 20), ("rows", 64, 1030, 12, 4),
                                                  ("rows", 256, 300, 16, 12)])
def test_many_sequences_of_a_row(name, D, B, R, width, i8):
    # as many rows as fill whole tiles, a row a sequence: 16-row tiles unless tables are short
    g = np.random.default_rng(B + width)
    ns = [int(x) for x in g.integers(0, 2, B)]
    lens = [int(x) for x in g.integers(0, 64 * width + 20, B) // (1 + 5 * (g.random(B) < 0.7))]
    path = {"items16": 2, "runs16": 4, "rows": 1}[name]
    f, c, table, q = kf.inputs(name, D, i8, 10, ns=ns, lens=lens, H=8, R=R, P=64, width=width, path=path)
    _check(name, f, c, table, q)
