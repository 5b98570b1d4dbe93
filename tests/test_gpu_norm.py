"""GPU parity of the residual's addition, norm and 8-bit rows: sums, scales and codes bit for bit
against the oracle (a row whose sum of squares lies next to a rounding border may be either of
two), and as it is called: in place, in wider buffers, captured, on two streams."""

import numpy as np
import pytest
import torch

import synthetic as syn
from gpu_util import DEV, assert_same, bf16_dev, dev, host, host_bf16_bits, poison
from oracle import layer
from oracle import numerics as nm

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq

KINDS = ("int8", "e4m3", "mx")
UNIT = {"int8": 16, "e4m3": 128, "mx": 32}
BLOCK = {"e4m3": 128, "mx": 32}


def _payload(kind):
    return {"int8": wq.WQ_PAYLOAD_INT8, "e4m3": wq.WQ_PAYLOAD_FP8_E4M3, "mx": wq.WQ_PAYLOAD_MXFP8}[kind]


def _wide(bits, pad):
    """The rows inside a wider buffer of NaN."""
    M, K = bits.shape
    buf = torch.full((M, K + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    buf[:, :K] = bf16_dev(bits)
    return buf[:, :K]


def _bf16_nan(v):
    """f32 -> bf16 bits; NaN as one pattern, values past the largest as infinity."""
    with np.errstate(over="ignore"):
        out = nm.f64_to_bf16_rn(np.where(np.isfinite(v), v, 0.0).astype(np.float64))
    out = np.where(np.isposinf(v), 0x7F80, np.where(np.isneginf(v), 0xFF80, out))
    return np.where(np.isnan(v), 0x7FC0, out).astype(np.uint16)


def _one_nan(bits):
    return np.where((bits & 0x7FFF) > 0x7F80, 0x7FC0, bits).astype(np.uint16)


def _rows(kind, v):
    if kind == "int8":
        return layer.rows_int8(v)
    codes, words = layer.rows_e4m3(v, BLOCK[kind])
    return codes[:, None], words


def _check(kind, x, r, gamma, *, eps=1e-6, pad=0, want_y=True):
    M, K = x.shape
    print(f"norm {kind} M={M} K={K} residual={r is not None} pad={pad}", flush=True)
    xd, rd, gd = _wide(x, pad), None if r is None else _wide(r, pad), bf16_dev(gamma)
    qshape, qtype = ((M, K), torch.int8) if kind == "int8" else ((M, 1, K), torch.uint8)
    packs = -(-K // (4 * BLOCK[kind])) if kind != "int8" else 0
    xs = poison((M,), torch.float32) if kind == "int8" else poison((1, packs, (M + 3) // 4 * 4), torch.int32)
    sums, y = poison((M, K + pad), torch.bfloat16), poison((M, K + pad), torch.bfloat16)
    got = wq.wq_add_rms_quant(xd, rd, gd, eps, payload=_payload(kind), x_q=poison(qshape, qtype), x_s=xs,
                              sum_out=sums[:, :K], y=y[:, :K] if want_y else None)
    torch.cuda.synchronize()
    h = x if r is None else layer.add_bf16(x, r)
    assert_same("sum", _one_nan(host_bf16_bits(sums[:, :K])), _one_nan(h))
    v, other = layer.normed(h, gamma, eps)
    codes, scale = _rows(kind, v)
    codes2, scale2 = _rows(kind, other)
    q, s = host(got[0]), host(got[1])
    yb, y1, y2 = _one_nan(host_bf16_bits(y[:, :K])), _one_nan(_bf16_nan(v)), _one_nan(_bf16_nan(other))
    for m in range(M):  # a row is one of its two readings, in all of its outputs
        fits = False
        for c, sc, yy in ((codes, scale, y1), (codes2, scale2, y2)):
            same_s = np.array_equal(s[m], sc[m], equal_nan=True) if kind == "int8" else np.array_equal(s[..., m], sc[..., m])
            fits |= np.array_equal(q[m], c[m]) and same_s and (not want_y or np.array_equal(yb[m], yy[m]))
        if not fits:
            assert_same(f"codes of row {m}", q[m].reshape(1, -1), codes[m].reshape(1, -1))
            assert_same(f"y of row {m}", yb[m][None], y1[m][None])
            raise AssertionError(f"row {m}: scales {s[..., m]} {scale[..., m]}")
    if kind != "int8":
        assert not s[..., M:].any()  # the padding words
    for buf in (sums, y) if want_y else (sums,):
        assert (host(buf[:, K:].contiguous().view(torch.int16)) == -0x5A5B).all()  # 0xA5A5: nothing behind the rows


def _inputs(seed, M, K, r=True):
    g = syn.rng(100, seed, M, K)
    x = syn.activations((101, seed, M, K), M, K)
    res = syn.activations((102, seed, M, K), M, K, outlier_frac=0.01, outlier_mul=30.0, row_scale=np.exp(g.standard_normal(M)))
    return x, res if r else None, nm.f64_to_bf16_rn(1 + 0.3 * g.standard_normal(K))


# widths on both sides of every rule between the kernel's forms, in units of each payload
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [16, 32, 128, 496, 512, 528, 640, 1152, 2048, 2064, 4096, 4224, 8192, 8320, 16384, 16512, 32768, 32896, 65536])
def test_widths(kind, K):
    K = -(-K // UNIT[kind]) * UNIT[kind]
    for M in (1, 2, 5):
        _check(kind, *_inputs(1, M, K), pad=8 if M == 2 else 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M, K", [(3, 4096), (64, 4096), (63, 1152), (257, 512), (1000, 256), (300, 2176), (600, 4096)])
def test_many_rows(kind, M, K):
    _check(kind, *_inputs(2, M, K), pad=16, want_y=M != 64)


# rows on either side of two for each CU, where a row has fewer threads
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [2176, 4096, 4224, 8192])
def test_as_many_rows_as_fill_the_chip(kind, K):
    most = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    for M in (most, most + 3):
        _check(kind, *_inputs(5, M, K), want_y=M > most)


@pytest.mark.parametrize("kind", KINDS)
def test_without_a_residual(kind):
    _check(kind, *_inputs(3, 5, 1152, r=False))
    xd, g = bf16_dev(_inputs(3, 5, 1152)[0]), bf16_dev(_inputs(3, 5, 1152)[2])
    assert wq.wq_add_rms_quant(xd, None, g, payload=_payload(kind))[2] is None


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_zeros_and_what_is_not_finite(kind):
    x, r, gamma = _inputs(4, 12, 1152)
    x[0], r[0] = 0, 0
    x[1], r[1] = 0x8000, 0x8000
    x[2, 5], r[3, 1151], x[4, 77], r[5, 300] = 0x7FC0, 0x7F80, 0xFF80, 0xFFC1
    x[6, 9], r[6, 9] = 0x7F7F, 0x7F7F          # their sum is an infinity
    x[7], r[7] = 0x0001, 0x8000                # subnormal
    x[8], r[8, :4] = 0x7F00, 0                 # the mean square beyond 32 bits
    _check(kind, x, r, gamma)
    gamma[3], gamma[700] = 0x7F80, 0x7FC0
    _check(kind, x, r, gamma)
    gamma[3], gamma[700], gamma[20] = 0, 0, 0x7F7F  # v beyond the largest
    _check(kind, x, r, gamma)
    _check(kind, x, r, gamma, eps=0.0)


@pytest.mark.parametrize("kind", KINDS)
def test_magnitudes_over_the_whole_range(kind):
    g = syn.rng(103)
    M, K = 24, 256
    x = nm.f64_to_bf16_rn(g.standard_normal((M, K)) * np.exp2(g.integers(-60, 60, (M, K)).astype(float)))
    r = nm.f64_to_bf16_rn(g.standard_normal((M, K)) * np.exp2(g.integers(-60, 60, (M, 1)).astype(float)))
    _check(kind, x, r, nm.f64_to_bf16_rn(np.exp2(g.integers(-20, 20, K).astype(float))))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [256, 4096, 16384])
def test_the_residual_stream_in_place(kind, K):
    x, r, gamma = _inputs(5, 33, K)
    xd, rd, gd = bf16_dev(x), bf16_dev(r), bf16_dev(gamma)
    want = wq.wq_add_rms_quant(xd, rd, gd, payload=_payload(kind), return_y=True)
    for name in ("residual", "x"):
        a, b = xd.clone(), rd.clone()
        to = b if name == "residual" else a
        got = wq.wq_add_rms_quant(a, b, gd, payload=_payload(kind), sum_out=to, return_y=True)
        assert got[2] is to and all(torch.equal(p.view(torch.uint8), w.view(torch.uint8)) for p, w in zip(got, want))
        other = a if name == "residual" else b
        assert torch.equal(other, xd if name == "residual" else rd)


def test_captured_on_streams_and_empty():
    x, r, gamma = _inputs(6, 40, 4096)
    xd, rd, gd = bf16_dev(x), bf16_dev(r), bf16_dev(gamma)
    kinds = [_payload(k) for k in KINDS]
    graph = torch.cuda.CUDAGraph()
    wq.wq_add_rms_quant(xd, rd, gd)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = [wq.wq_add_rms_quant(xd, rd, gd, payload=p) for p in kinds]
    for i in range(3):
        rd.copy_(bf16_dev(_inputs(7 + i, 40, 4096)[1]))
        graph.replay()
        eager = [wq.wq_add_rms_quant(xd, rd, gd, payload=p) for p in kinds]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, e in zip(outs, eager) for a, b in zip(o, e))
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(4):
        for st, p in zip(streams, kinds):
            with torch.cuda.stream(st):
                got.append(wq.wq_add_rms_quant(xd, rd, gd, payload=p))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i, o in enumerate(got) for a, b in zip(o, eager[i % 2]))
    q, s, h = wq.wq_add_rms_quant(xd[:0], rd[:0], gd)
    assert q.shape == (0, 4096) and s.shape == (0,) and h.shape == (0, 4096)


@pytest.mark.parametrize("kind", KINDS)
def test_the_products_read_it(kind):
    """Rows from the norm through the product are the product of what the codes stand for."""
    M, K, N = 17, 1024, 128
    x, r, gamma = _inputs(9, M, K)
    q, s, _ = wq.wq_add_rms_quant(bf16_dev(x), bf16_dev(r), bf16_dev(gamma), payload=_payload(kind))
    g = syn.rng(104)
    if kind == "int8":
        w, sw = g.integers(-127, 128, (N, K)).astype(np.int8), np.full(N, 2.0**-10, np.float32)
        y = wq.wq_quant_matmul(q, s, dev(w), dev(sw))
        want = (host(q).astype(np.float64) @ w.T) * host(s).astype(np.float64)[:, None] * 2.0**-10
    else:
        from oracle import fp8_group as fg

        codes = (g.integers(0, 0x57, (1, N, K)) | (g.integers(0, 2, (1, N, K)) << 7)).astype(np.uint8)
        if kind == "e4m3":
            y = wq.wq_quant_matmul(q, s, dev(codes), torch.full((1, N // 128, K // 128), 2.0**-4, device=DEV), fp8_groups=1)
        else:
            y = wq.wq_quant_matmul(q, s, dev(codes), torch.full((1, N, K // 32), 127 - 4, dtype=torch.uint8, device=DEV), fp8_groups=1, mx=True)
        block = BLOCK[kind]
        e = fg.unpack_ue8m0(host(s), M, K // block)[:, 0].astype(int) - 127
        a = nm.e4m3_decode(host(q)[:, 0]) * np.repeat(np.exp2(e.astype(float)), block, 1)
        want = (a @ nm.e4m3_decode(codes[0]).T) * 2.0**-4
        y = y[:, 0]
    got = nm.bf16_to_f32(host_bf16_bits(y)).astype(np.float64)
    # one rounding to bf16 (2^-8) and the matrix unit's sums in f32 with its alignment (well below 2^-10
    # of the largest of K products of alike size, whose sum these random signs do not cancel far)
    scale = np.abs(want).max(1, keepdims=True)
    assert (np.abs(got - want) <= 2.0**-8 * np.abs(want) + 2.0**-10 * scale).all()
