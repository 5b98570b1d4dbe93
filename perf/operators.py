"""The library's 4-bit microscaled operators and its 8-bit paged cache, as measured cases.

Four kinds of case:
  quant   bf16 rows -> E2M1 codes with a UE8M0 scale for 32 elements, and the values they stand for
  product y = A W^T over those blocks: 4-bit (w4a4) or E4M3 (w4a8) activations, 4-bit weights
  append  new k and v rows quantised into a paged 8-bit cache (a scale for each page and head)
  attend  attention of q rows over that cache, from one row a sequence to whole prompts

With ``own`` false ``run`` computes the plain form in elementary torch operations, otherwise it
calls the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
# E2M1 values by code: sign, two exponent bits (bias 1), one fraction bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
# mantissa (of [0.5, 1)) and exponent of each format's largest magnitude: 6, 448, 127
TOP = {"e2m1": (0.75, 3), "e4m3": (0.875, 9), "int8": (0.9921875, 7)}


# ---- cases ---------------------------------------------------------------------------------------


def listed():
    return [
        # one decoded token's attention output before the grouped output projection
        dict(name="quant_token", op="quant", T=1, G=8, D=4096),
        # a long prompt's hidden rows before a 4-bit projection
        dict(name="quant_prompt", op="quant", T=8192, G=1, D=4096),
        # one decoded token through the down projection of the query, 4-bit on both sides: latency
        dict(name="product_token", op="product", a="e2m1", M=1, G=1, N=1024, K=4096, pad=0),
        # a decode batch through the grouped output projection, 8-bit activations on 4-bit weights
        dict(name="product_groups", op="product", a="e4m3", M=64, G=8, N=1024, K=4096, pad=0),
        # an odd chunk of a prompt, rows inside a wider buffer
        dict(name="product_ragged", op="product", a="e4m3", M=1000, G=1, N=2064, K=1152, pad=64),
        # a prompt through the wide query projection: the largest product
        dict(name="product_prompt", op="product", a="e2m1", M=8192, G=1, N=32768, K=1024, pad=0),
        # one new token for each of 64 running sequences
        dict(name="append_decode", op="append", code="int8", B=64, n=1, L=1000, H=8, D=128, P=64),
        # three prompts of different lengths written at once, one behind a cached prefix
        dict(name="append_prompt", op="append", code="e4m3", B=3, n=2000, L=2500, H=8, D=128, P=32),
        # one sequence, one token: latency
        dict(name="attend_token", op="attend", code="e4m3", B=1, n=1, L=1000, H=8, R=4, D=128, P=16, causal=True),
        # a ragged decode batch: bandwidth
        dict(name="attend_batch", op="attend", code="int8", B=64, n=1, L=8192, H=8, R=4, D=128, P=64, causal=True),
        # one very long sequence with one shared head of keys, four drafted tokens at once
        dict(name="attend_long", op="attend", code="e4m3", B=1, n=4, L=131072, H=1, R=16, D=256, P=128, causal=True),
        # two chunks of prompts behind cached prefixes: arithmetic
        dict(name="attend_prompt", op="attend", code="e4m3", B=2, n=2000, L=4099, H=8, R=4, D=128, P=64, causal=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "product", "append", "attend"))
    if op == "quant":
        G = rng.choice((1, 2, 3, 8))
        D = 32 * _spread(rng, 1, 256)
        return dict(op=op, T=_spread(rng, 1, max(1, min(8192, (8192 * 4096) // (G * D)))), G=G, D=D)
    if op == "product":
        a = rng.choice(("e2m1", "e4m3"))
        G, K = rng.choice((1, 1, 2, 8)), 128 * _spread(rng, 1, 64)
        N = 16 * _spread(rng, 4, min(2048, 65536 * 4096 // (16 * G * K)))
        M = _spread(rng, 1, min(8192, max(1, 8192 * 32768 * 1024 // (G * N * K)), 8192 * 32768 // (G * N)))
        return dict(op=op, a=a, M=M, G=G, N=N, K=K, pad=rng.choice((0, 16, 64)))
    code, D = rng.choice(("e4m3", "int8")), rng.choice((64, 128, 256))
    P, H, B = rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 3, 4, 8)), _spread(rng, 1, 128)
    if op == "append":
        n = _spread(rng, 1, max(2, 6000 * 1024 // (B * H * D)))
        before = _spread(rng, 1, max(2, min(2000, 40_000_000 // (B * H * D))))
        return dict(op=op, code=code, B=B, n=n, L=n + before, H=H, D=D, P=P)
    L = _spread(rng, 1, max(2, min(131072, 64 * 8192 * 1024 // (B * H * D))))
    R = rng.choice((1, 2, 4, 5, 8, 16))
    n = _spread(rng, 1, max(1, min(L, 4000, 2 * 2000 * 4099 * 4096 // (B * L * H * R * D))))
    return dict(op=op, code=code, B=B, n=n, L=L, H=H, R=R, D=D, P=P, causal=rng.random() < 0.8)


def _lengths(case):
    """New rows and whole length of each sequence: the first has both at their largest, the others less."""
    B, n, L = case["B"], case["n"], case["L"]
    new, whole = [], []
    for b in range(B):
        new.append(n if b == 0 else max(1, n - (n * (7 * b % 16)) // 20))
        whole.append(L if b == 0 else max(new[b], L - (L * (5 * b % 32)) // 34))
    return new, whole


def _pairs(case):
    """Keys that the rows of all sequences see, in all."""
    seen = 0
    for n, whole in zip(*_lengths(case)):
        seen += sum(whole - n + i + 1 for i in range(n)) if case["causal"] else n * whole
    return seen


def work(case):
    if case["op"] == "quant":
        n = case["T"] * case["G"] * case["D"]
        return {"bytes": 2 * n + n / 2 + n / 32 + 2 * n, "flops": 0}
    if case["op"] == "product":
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        a = M * G * (K / 2 if case["a"] == "e2m1" else K) + M * G * K / 32
        return {"bytes": a + G * N * (K / 2 + K / 32) + 2 * M * G * N, "flops": 2 * M * G * N * K}
    new, whole = _lengths(case)
    row = case["H"] * case["D"]
    if case["op"] == "append":
        return {"bytes": sum(new) * row * (4 + 2), "flops": 0}
    q = sum(new) * row * case["R"]
    return {"bytes": 2 * sum(whole) * row + 4 * q, "flops": 4 * _pairs(case) * row * case["R"]}


# ---- the formats, in torch -------------------------------------------------------------------------


def _exponent(a, code):
    """The smallest e with 2^e >= a / (the format's largest magnitude), at least -127."""
    m, k = torch.frexp(a)
    top, shift = TOP[code]
    e = k - shift + (m > top).to(k.dtype)
    return torch.where(a > 0, e, torch.full_like(e, -127)).clamp_(min=-127)


def _round_e2m1(y):
    """f32 values within 6 -> the E2M1 code of the nearest, ties to the even code."""
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.round(a / step) * step
    c = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r / 2 + 4))
    return c.to(torch.uint8) + 8 * torch.signbit(y).to(torch.uint8)


def _pair_nibbles(codes):
    c = codes.view(*codes.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4)


def _nibbles(pairs):
    return torch.stack((pairs & 15, pairs >> 4), dim=-1).flatten(-2)


def _pack_bytes(byte):
    """Scale bytes [T, G, blocks] -> int32 words [G, ceil(blocks / 4), 4 ceil(T / 4)]."""
    T, G, h = byte.shape
    full = torch.zeros((-(-T // 4) * 4, G, -(-h // 4) * 4), dtype=torch.uint8, device=byte.device)
    full[:T, :, :h] = byte
    return full.view(full.shape[0], G, -1, 4).permute(1, 2, 0, 3).contiguous().view(torch.int32).squeeze(-1)


def _scales(words, T):
    """int32 words [G, packs, tokens] -> f32 powers of two [T, G, 4 packs]."""
    G, ph, ta = words.shape
    b = words.view(torch.uint8).view(G, ph, ta, 4)[:, :, :T].permute(2, 0, 1, 3).reshape(T, G, ph * 4)
    return torch.ldexp(torch.ones((), device=b.device), b.to(torch.int32) - 127)


def _blocks_of(x, code):
    """f32 [T, G, D] -> codes (one a byte) and scale words, 32 elements to a scale."""
    T, G, D = x.shape
    v = x.view(T, G, D // 32, 32)
    e = _exponent(v.abs().amax(-1), code)
    y = torch.ldexp(v, -e[..., None]).view(T, G, D)
    q = _round_e2m1(y) if code == "e2m1" else y.to(torch.float8_e4m3fn).view(torch.uint8)
    return q, _pack_bytes((e + 127).to(torch.uint8))


def _values(q, words, code):
    """Codes and scale words -> f32 [T, G, D]."""
    if code == "e2m1":
        v = torch.tensor(E2M1, device=q.device)[_nibbles(q).to(torch.int32)]
    else:
        v = q.view(torch.float8_e4m3fn).float()
    T, G, D = v.shape
    s = _scales(words, T)[:, :, : D // 32]
    return (v.view(T, G, D // 32, 32) * s[..., None]).view(T, G, D)


def _as_values(codes):
    """Cache codes as the numbers they stand for: int8 numbers or E4M3 values."""
    return codes if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn)


# ---- inputs ---------------------------------------------------------------------------------------


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _cache(gen, case, pages):
    """A filled cache: k [pages, H, P, D], v [pages, H, D, P], scale bytes [pages, H]."""
    H, D, P, code = case["H"], case["D"], case["P"], case["code"]
    kind = torch.int8 if code == "int8" else torch.uint8
    k = torch.empty((pages, H, P, D), dtype=kind, device=DEV)
    v = torch.empty((pages, H, D, P), dtype=kind, device=DEV)
    ks = torch.empty((pages, H), dtype=torch.uint8, device=DEV)
    vs = torch.empty((pages, H), dtype=torch.uint8, device=DEV)
    # keys have a few large channels, as rotary attention's do
    channel = 1 + 4 * (torch.rand((H, 1, D), generator=gen, device=DEV) < 0.05)
    part = max(1, (1 << 26) // (H * D * P))
    for at in range(0, pages, part):
        to = min(pages, at + part)
        for side in (0, 1):
            x = _normal(gen, to - at, H, P, D)
            if side == 0:
                x *= channel
            e = _exponent(x.abs().amax((-1, -2)), code)
            y = torch.ldexp(x, -e[..., None, None])
            y = y.round_().to(torch.int8) if code == "int8" else y.to(torch.float8_e4m3fn).view(torch.uint8)
            if side == 0:
                k[at:to], ks[at:to] = y, (e + 127).to(torch.uint8)
            else:
                v[at:to], vs[at:to] = y.transpose(-1, -2), (e + 127).to(torch.uint8)
    return k, v, ks, vs


def _paged(gen, case):
    """Row offsets, lengths and a table that gives every sequence pages in no order."""
    new, whole = _lengths(case)
    P = case["P"]
    need = [-(-w // P) for w in whole]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((case["B"], max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at : at + c]
        at += c
    offsets = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int64, device=DEV)
    return pages, table, offsets, torch.tensor(whole, dtype=torch.int32, device=DEV), new, whole


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "quant":
        T, G, D = case["T"], case["G"], case["D"]
        x = _normal(gen, T, G, D) * torch.exp(_normal(gen, T, 1, 1))
        s["x"] = x.bfloat16()
        return s
    if case["op"] == "product":
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        a, sa = _blocks_of(_normal(gen, M, G, K) * torch.exp(0.5 * _normal(gen, M, 1, 1)), case["a"])
        a = _pair_nibbles(a) if case["a"] == "e2m1" else a
        wide = torch.zeros((M, G, a.shape[2] + case["pad"]), dtype=torch.uint8, device=DEV)
        wide[:, :, : a.shape[2]] = a
        w, sw = [], []
        for _ in range(G):  # weights are cast group by group: a group is [N, 1, K]
            q, words = _blocks_of(_normal(gen, N, 1, K) * K**-0.5, "e2m1")
            w.append(_pair_nibbles(q).view(N, K // 2))
            sw.append(words)
        s.update(a=wide[:, :, : a.shape[2]], sa=sa, w=torch.stack(w), sw=torch.cat(sw))
        return s
    pages, table, offsets, lens, new, whole = _paged(gen, case)
    s["k"], s["v"], s["ks"], s["vs"] = _cache(gen, case, pages)
    s.update(table=table, offsets=offsets, lens=lens, new=new, whole=whole)
    rows, H, D, P = sum(new), case["H"], case["D"], case["P"]
    if case["op"] == "append":
        # some rows are larger than what their page holds: its scale has to grow
        loud = torch.exp2(torch.randint(-1, 3, (rows, 1, 1), generator=gen, device=DEV).float())
        s["kn"], s["vn"] = ((_normal(gen, rows, H, D) * loud).bfloat16() for _ in range(2))
        # the pages that the new rows fall in: the scheduler that gave them out knows them
        s["touched"] = torch.cat([table[b, (w - n) // P : -(-w // P)] for b, (n, w) in enumerate(zip(new, whole))]).long()
    else:
        s["q"] = (_normal(gen, rows, H * case["R"], D)).bfloat16()
        s["most"] = (max(new), max(whole))  # as a scheduler knows them
    return s


# ---- one pass -------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if op == "quant":
        return {"values": _own_quant(s) if own else _plain_quant(s)}
    if op == "product":
        return {"y": _own_product(s) if own else _plain_product(s)}
    if op == "append":
        _own_append(s) if own else _plain_append(s)
        scales = {"k_scale": s["ks"].view(torch.float8_e8m0fnu), "v_scale": s["vs"].view(torch.float8_e8m0fnu)}
        return {"k": _as_values(s["k"]), "v": _as_values(s["v"]), **scales}
    out, lse = _own_attend(s) if own else _plain_attend(s)
    return {"out": out, "lse": lse}


def _own_quant(s):
    import fp8_dynamic_quant_amd as wq

    q, _, words = wq.wq_group_quant_mxfp4(s["x"])
    return wq.wq_group_dequant_mxfp4(q, words)


def _own_product(s):
    import fp8_dynamic_quant_amd as wq

    return wq.wq_quant_matmul(s["a"], s["sa"], s["w"], s["sw"], fp8_groups=s["case"]["G"], mx4=True)


def _own_append(s):
    import fp8_dynamic_quant_amd as wq

    cache = wq.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    wq.wq_kv_append(cache, s["kn"], s["vn"], s["offsets"], s["lens"], s["table"])


def _own_attend(s):
    import fp8_dynamic_quant_amd as wq

    cache = wq.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    return wq.wq_kv_attention(cache, s["q"], s["offsets"], s["lens"], s["table"], causal=s["case"]["causal"],
                              return_lse=True)


def _plain_quant(s):
    q, words = _blocks_of(s["x"].float(), "e2m1")
    return _values(_pair_nibbles(q), words, "e2m1").bfloat16()


def _plain_product(s):
    a = _values(s["a"].contiguous(), s["sa"], s["case"]["a"])
    w = _values(s["w"].transpose(0, 1).contiguous(), s["sw"], "e2m1")
    return torch.matmul(a.transpose(0, 1), w.permute(1, 2, 0)).transpose(0, 1).bfloat16()


def _row_places(s):
    """Sequence, index among its new rows and position of every row."""
    r = torch.arange((s["kn"] if "kn" in s else s["q"]).shape[0], device=DEV)
    b = torch.searchsorted(s["offsets"], r, right=True) - 1
    i = r - s["offsets"][b]
    n = s["offsets"][b + 1] - s["offsets"][b]
    return b, i, s["lens"][b] - n + i


def _plain_append(s):
    code, P = s["case"]["code"], s["case"]["P"]
    b, _, at = _row_places(s)
    page, slot = s["table"][b, at // P].long(), at % P
    touched = s["touched"]
    # the first new slot of every page: what stands before it is kept, at the page's new scale
    first = torch.full((s["ks"].shape[0],), P, device=DEV).scatter_reduce_(0, page, slot, "amin")[touched]
    kept, before = first[:, None] > 0, (torch.arange(P, device=DEV) < first[:, None])[:, None]

    def put(codes, scale, x, columns):
        x = x.float()
        most = torch.zeros(scale.shape, device=DEV)
        most.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
        new, old = _exponent(most[touched], code), scale[touched].int() - 127
        e = torch.where(kept, torch.maximum(old, new), new)
        shift = torch.where(kept, old - e, torch.zeros_like(e))
        scale[touched] = (e + 127).to(torch.uint8)
        at_row = scale[page].int() - 127
        y = torch.ldexp(x, -at_row[..., None])
        held = codes[touched]
        shift = (shift[..., None] * before)[:, :, None] if columns else (shift[..., None] * before)[..., None]
        if code == "int8":
            held = torch.round(torch.ldexp(held.float(), shift)).to(torch.int8)
            y = torch.round(y).to(torch.int8)
        else:
            held = torch.ldexp(held.view(torch.float8_e4m3fn).float(), shift)
            held, y = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (held, y))
        codes[touched] = held
        if columns:
            codes[page, :, :, slot] = y
        else:
            codes[page, :, slot] = y

    put(s["k"], s["ks"], s["kn"], False)
    put(s["v"], s["vs"], s["vn"], True)


def _plain_attend(s):
    case = s["case"]
    B, H, R, D, P = case["B"], case["H"], case["R"], case["D"], case["P"]
    b, i, _ = _row_places(s)
    most_new, most = s["most"]
    table = s["table"].long()

    def gather(codes, scale):
        x = codes[table] if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn)[table]
        return x.float() * torch.ldexp(torch.ones((), device=DEV), scale[table].int() - 127)[..., None, None]

    k = gather(s["k"], s["ks"]).transpose(1, 2).reshape(B, H, -1, D)[:, :, :most]
    v = gather(s["v"], s["vs"]).permute(0, 2, 1, 4, 3).reshape(B, H, -1, D)[:, :, :most]
    q = torch.zeros((B, most_new, H, R, D), device=DEV)
    q[b, i] = s["q"].float().view(-1, H, R, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, most_new * R, D)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(D**-0.5).view(B, H, most_new, R, most)
    j = torch.arange(most, device=DEV)
    last = s["lens"][:, None].expand(B, most_new) - 1
    if case["causal"]:
        n = s["offsets"][1:] - s["offsets"][:-1]
        last = last - n[:, None] + 1 + torch.arange(most_new, device=DEV)
    hide = j > last[:, None, :, None, None]
    score.masked_fill_(hide, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    some = total > 0
    lse = torch.where(some, top + total.log(), torch.full_like(top, float("-inf")))
    o = torch.matmul(p.view(B, H, most_new * R, most), v).view(B, H, most_new, R, D)
    o = torch.where(some, o / torch.where(some, total, torch.ones_like(total)), torch.zeros_like(o))
    out = o.permute(0, 2, 1, 3, 4)[b, i].reshape(-1, H * R, D).bfloat16()
    return out, lse.permute(0, 2, 1, 3, 4)[b, i].reshape(-1, H * R)


# ---- the definition in 64 bits ---------------------------------------------------------------------


def _power64(e):
    return np.ldexp(1.0, e.astype(np.int64))


def _block_exponent64(a, largest):
    """Smallest e >= -127 with largest * 2^e >= a, by comparisons."""
    e = np.full(a.shape, -127, dtype=np.int64)
    for step in (128, 64, 32, 16, 8, 4, 2, 1):
        # the largest e that is still too small, then one more
        e = np.where(np.ldexp(largest, e + step - 1) < a, e + step, e)
    return e


def _nearest64(y, grid):
    """The nearest value of a sorted grid of magnitudes; between two, the one at the even index."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    d = (a - grid[lo]) - (grid[hi] - a)
    at = np.where(d < 0, lo, np.where(d > 0, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(grid[at], y)


GRID_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
GRID_E4M3 = np.array([m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def _host(t):
    return t.detach().to("cpu").double().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = _host(s["x"].float())
        v = x.reshape(*x.shape[:2], -1, 32)
        e = _block_exponent64(np.abs(v).max(-1), 6.0)[..., None]
        y = _nearest64(v * _power64(-e), GRID_E2M1) * _power64(e)
        return {"values": torch.from_numpy(y.reshape(x.shape))}
    if case["op"] == "product":
        return {"y": _exact_product(s, case)}
    if case["op"] == "append":
        return _exact_append(s, case)
    return _exact_attend(s, case)


def _decode64(codes, kind):
    """E2M1 pairs or E4M3 bytes -> f64, from the fields of a code."""
    c = codes.to(torch.int64)
    if kind == "e2m1":
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)
        sign, ef, f, bias, width = c // 8, c // 2 % 4, c % 2, 1, 1
    else:
        sign, ef, f, bias, width = c // 128, c // 8 % 16, c % 8, 7, 3
    f = f.double() / 2**width
    v = torch.where(ef == 0, f * 2.0 ** (1 - bias), (1 + f) * torch.pow(2.0, (ef - bias).double()))
    return v * (1 - 2 * sign)


def _exact_product(s, case):
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    y = torch.empty((M, G, N), dtype=torch.float64, device=DEV)

    def scaled(codes, words, rows, kind):
        v = _decode64(codes, kind)
        w = words[:, :rows].long()  # [K / 128, rows]
        e = torch.stack([w >> sh & 255 for sh in (0, 8, 16, 24)], -1)  # [K / 128, rows, 4]
        e = e.transpose(0, 1).reshape(rows, -1)[:, : K // 32]
        return (v.view(rows, K // 32, 32) * torch.pow(2.0, (e - 127).double())[..., None]).view(rows, K)

    for g in range(G):
        a = scaled(s["a"][:, g].contiguous(), s["sa"][g], M, case["a"])
        w = scaled(s["w"][g], s["sw"][g], N, "e2m1")
        y[:, g] = a @ w.t().contiguous()
    return y


def _exact_append(s, case):
    H, P, code = case["H"], case["P"], case["code"]
    table = _host(s["table"])
    out = {}
    for side, transposed in (("k", False), ("v", True)):
        held = s[side]
        held = _host(held.double()) if code == "int8" else _host(_decode64(held, "e4m3"))
        held = held.swapaxes(-1, -2).copy() if transposed else held
        e = _host(s[side + "s"]).astype(np.int64) - 127
        x, row = _host(s[side + "n"].float()), 0
        for b, (n, whole) in enumerate(zip(s["new"], s["whole"])):
            for at in range((whole - n) // P, -(-whole // P)):
                lo, hi = max(whole - n, at * P), min(whole, (at + 1) * P)
                part = x[row : row + hi - lo].swapaxes(0, 1)  # [H, rows, D]
                row += hi - lo
                page, slot = table[b, at], lo - at * P
                en = _block_exponent64(np.abs(part).max((-1, -2)), 127.0 if code == "int8" else 448.0)
                if slot > 0:
                    en = np.maximum(en, e[page])
                    old = held[page][:, :slot] * _power64(e[page] - en)[:, None, None]
                    held[page, :, :slot] = np.rint(old) if code == "int8" else _nearest64(old, GRID_E4M3)
                # slots behind the new rows keep their codes
                y = part * _power64(-en)[:, None, None]
                held[page, :, slot : slot + hi - lo] = np.rint(y) if code == "int8" else _nearest64(y, GRID_E4M3)
                e[page] = en
        held = held.swapaxes(-1, -2).copy() if transposed else held
        out[side] = torch.from_numpy(held.astype(np.int8) if code == "int8" else held)
        out[side + "_scale"] = torch.from_numpy(_power64(e))
    return out


def _exact_attend(s, case):
    H, R, D, P = case["H"], case["R"], case["D"], case["P"]
    if _pairs(case) * H * R * D > 3e12:
        return None
    q, rows = s["q"].double(), s["q"].shape[0]
    out = torch.zeros((rows, H * R, D), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, H * R), -math.inf, dtype=torch.float64, device=DEV)

    def of_head(codes, scale, pages, h):
        c = codes[pages, h]
        c = c.double() if code == "int8" else _decode64(c, "e4m3")
        return c * torch.pow(2.0, scale[pages, h].double() - 127)[:, None, None]

    code, row = case["code"], 0
    for b, (n, whole) in enumerate(zip(s["new"], s["whole"])):
        pages = s["table"][b, : -(-whole // P)].long()
        for h in range(H):
            k = of_head(s["k"], s["ks"], pages, h).reshape(-1, D)[:whole]
            v = of_head(s["v"], s["vs"], pages, h).transpose(1, 2).reshape(-1, D)[:whole]
            for r in range(R):
                z = (q[row : row + n, h * R + r] @ k.t().contiguous()) / math.sqrt(D)
                if case["causal"]:
                    z = z + torch.full_like(z, -math.inf).triu(whole - n + 1)
                lse[row : row + n, h * R + r] = torch.logsumexp(z, -1)
                out[row : row + n, h * R + r] = torch.softmax(z, -1) @ v
        row += n
    return {"out": out, "lse": lse}
