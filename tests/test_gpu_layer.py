"""A layer's attention half as a server runs it, call after call: the residual's norm in 8 bits, the
product to queries, keys and values, those turned on their way into the cache, attention behind what
the sequences share, the product back, the next norm.  Every stage against the oracle on the bytes
that the stage before left; a prompt, questions of several tokens and single tokens; captured."""

import numpy as np
import pytest
import torch

import kv_forms as kf
import synthetic as syn
from gpu_util import DEV, assert_same, bf16_dev, dev, host, host_bf16_bits
from oracle import int8_linear, layer
from oracle import numerics as nm
from test_gpu_shared import _limits

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq

K, H, R, P, WIDTH = 512, 2, 4, 32, 8
SHARED = 128
# (new tokens of each of the five sequences, lengths behind them): the shared prompt into the first
# one's pages, questions of different lengths and none, a token each but of the last
STEPS = [([128, 0, 0, 0, 0], [128, 0, 0, 0, 0]), ([9, 20, 1, 37, 0], [137, 148, 129, 165, 0]), ([1, 1, 1, 1, 0], [138, 149, 130, 166, 0])]


class _Layer:
    def __init__(self, D, i8):
        self.D, self.i8, self.Hq = D, i8, H * R
        N = (self.Hq + 2 * H) * D
        # (weights of gain one: queries and keys near one, whose scores _limits takes)
        (self.w, self.sw), (self.wo, self.swo) = (
            (w, (1 / np.sqrt((w.astype(np.float64) ** 2).sum(1))).astype(np.float32))
            for w in (syn.int8_weights((130, D), N, K)[0], syn.int8_weights((131, D), K, self.Hq * D)[0]))
        g = syn.rng(132, D, int(i8))
        self.g = g
        self.gamma = [nm.f64_to_bf16_rn(1 + 0.1 * g.standard_normal(K)) for _ in range(2)]
        pages = 5 * WIDTH + 1
        self.c = list(kf.cache(g, pages, H, P, D, i8))
        self.table = g.permutation(pages)[: 5 * WIDTH].reshape(5, WIDTH).astype(np.int32)
        self.table[1:, : SHARED // P] = self.table[0, : SHARED // P]
        self.group, self.shared = [0] * 5, [SHARED] * 5
        self.d = dict(w=dev(self.w), sw=dev(self.sw), wo=dev(self.wo), swo=dev(self.swo), gamma=[bf16_dev(x) for x in self.gamma],
                      cache=wq.KvCache(*(dev(x) for x in self.c)), table=dev(self.table), angles=wq.rotary_angles(WIDTH * P, D, device=DEV),
                      group=dev(np.array(self.group, np.int32)), shared=dev(np.array(self.shared, np.int32)))

    def rows(self, T):
        return [nm.f64_to_bf16_rn(self.g.standard_normal((T, K)) * s) for s in (1.0, 2.0)]

    def run(self, x, residual, off, lens):
        """Every stage's outputs, by name."""
        d, D, T, Hq = self.d, self.D, x.shape[0], self.Hq
        xq, xs, h = wq.wq_add_rms_quant(x, residual, d["gamma"][0])
        qkv = wq.wq_quant_matmul(xq, xs, d["w"], d["sw"]).view(T, Hq + 2 * H, D)
        before = qkv.clone()
        q, k, v = qkv[:, :Hq], qkv[:, Hq : Hq + H], qkv[:, Hq + H :]
        wq.wq_kv_append_rotated(d["cache"], k, v, off, lens, d["table"], d["angles"], q=q, q_out=q)
        out, lse = wq.wq_kv_attention_shared(d["cache"], q, off, lens, d["table"], d["group"], d["shared"], return_lse=True)
        aq, sa = wq.wq_dynamic_quant(out.view(T, Hq * D))
        y = wq.wq_quant_matmul(aq, sa, d["wo"], d["swo"])
        yq, ys, h2 = wq.wq_add_rms_quant(y, h, d["gamma"][1])
        return dict(xq=xq, xs=xs, h=h, before=before, qkv=qkv, out=out, lse=lse, aq=aq, sa=sa, y=y, yq=yq, ys=ys, h2=h2)


def _norm_is(name, x, r, gamma, codes, scales, total):
    h = layer.add_bf16(x, r)
    assert_same(name + " sum", host_bf16_bits(total), h)
    either = [layer.rows_int8(v) for v in layer.normed(h, gamma)]
    got = host(codes), host(scales)
    same = [(got[0] == q).all(1) & (got[1].view(np.uint32) == s.view(np.uint32)) for q, s in either]
    assert (same[0] | same[1]).all(), (name, np.flatnonzero(~(same[0] | same[1]))[:5])


def _product_is(name, q, s, w, sw, got):
    # the epilogue as it is documented: two products in f32, each rounded, and one rounding to bf16
    acc = int8_linear.gemm_int8_int32(host(q), w).astype(np.float32)
    want = nm.f64_to_bf16_rn(((acc * host(s)[:, None]) * sw[None].astype(np.float32)).astype(np.float64))
    assert_same(name, host_bf16_bits(got), want)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_layer_stage_by_stage(D, i8):
    m = _Layer(D, i8)
    for ns, lens in STEPS:
        off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
        T = int(off[-1])
        x, r = m.rows(T)
        print(f"layer D={D} i8={i8} n={ns} lens={lens}", flush=True)
        o = m.run(bf16_dev(x), bf16_dev(r), dev(off), dev(np.array(lens, np.int32)))
        torch.cuda.synchronize()
        _norm_is("first norm", x, r, m.gamma[0], o["xq"], o["xs"], o["h"])
        _product_is("q, k, v", o["xq"], o["xs"], m.w, m.sw, o["before"].view(T, -1))
        raw = host_bf16_bits(o["before"])
        angles = host(m.d["angles"])
        turned = layer.turned(nm.bf16_to_f32(raw[:, : m.Hq]), layer.positions_of(off, lens), angles, False)
        q = nm.f64_to_bf16_rn(turned.astype(np.float64))
        assert_same("q", host_bf16_bits(o["qkv"][:, : m.Hq]), q)
        layer.append_rotated(*m.c, raw[:, m.Hq : m.Hq + H], raw[:, m.Hq + H :], angles, False, off, lens, m.table)
        for name, got, want in zip(("k", "v", "k_scale", "v_scale"), m.d["cache"], m.c):
            assert_same(name, host(got), want)
        want, want_lse, mag, smag = kf.attention(m.c, q, off, lens, m.table, D**-0.5, True)
        lim, lim_lse = _limits(want, want_lse, mag, smag, max(lens), D)
        assert (np.abs(nm.bf16_to_f32(host_bf16_bits(o["out"])) - want) <= lim).all()
        assert (np.abs(host(o["lse"]) - want_lse) <= lim_lse).all()
        aq, sa = int8_linear.quant_int8_per_token(host_bf16_bits(o["out"]).reshape(T, -1))
        assert_same("attention's codes", host(o["aq"]), aq)
        assert_same("attention's scales", host(o["sa"]), sa)
        _product_is("y", o["aq"], o["sa"], m.wo, m.swo, o["y"])
        _norm_is("second norm", host_bf16_bits(o["y"]), host_bf16_bits(o["h"]), m.gamma[1], o["yq"], o["ys"], o["h2"])


@pytest.mark.parametrize("D, i8", [(64, True), (128, False), (256, False)])
def test_a_layer_captured(D, i8):
    m = _Layer(D, i8)
    for ns, lens in STEPS[:2]:
        off = np.concatenate(([0], np.cumsum(ns))).astype(np.int64)
        m.run(*(bf16_dev(x) for x in m.rows(int(off[-1]))), dev(off), dev(np.array(lens, np.int32)))
    ns, lens = STEPS[2]
    off = dev(np.concatenate(([0], np.cumsum(ns))).astype(np.int64))
    lens = dev(np.array(lens, np.int32))
    x, r = (bf16_dev(v) for v in m.rows(4))
    torch.cuda.synchronize()
    start = [t.clone() for t in m.d["cache"]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.run(x, r, off, lens)
    names = ("xq", "xs", "h", "qkv", "out", "lse", "y", "yq", "ys", "h2")
    for i in range(4):  # a token more each time, in the graph and then eagerly from the same cache
        for t, v in zip((x, r), m.rows(4)):
            t.copy_(bf16_dev(v))
        graph.replay()
        torch.cuda.synchronize()
        graphs = [t.clone() for t in m.d["cache"]] + [got[n].clone() for n in names]
        for t, v in zip(m.d["cache"], start):
            t.copy_(v)
        eager = m.run(x, r, off, lens)
        torch.cuda.synchronize()
        for a, b in zip(graphs, [*m.d["cache"]] + [eager[n] for n in names]):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        start = [t.clone() for t in m.d["cache"]]
        lens += torch.tensor([1, 1, 1, 1, 0], dtype=torch.int32, device=DEV)
