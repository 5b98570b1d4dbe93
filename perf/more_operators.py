"""What surrounds the library's products and its paged cache in a layer, as measured cases.

Three kinds of case:
  norm    the residual's addition, the root-mean-square norm of the sum, and its rows in 8 bits
          with scales (int8 a row, E4M3 with a scale for 128 elements or for 32)
  rotate  new k and v rows appended to the paged 8-bit cache, keys and queries turned by their
          positions on the way
  shared  attention over that cache of sequences that begin with the same pages

With ``own`` false ``run`` computes the plain form in elementary torch operations, otherwise it
calls the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
# mantissa (of [0.5, 1)) and exponent of each format's largest magnitude: 448, 127
TOP = {"e4m3": (0.875, 9), "int8": (0.9921875, 7)}
BLOCK = {"e4m3": 128, "mx": 32}


# ---- cases ---------------------------------------------------------------------------------------


def listed():
    return [
        # one decoded token in front of an int8 projection: latency
        dict(name="norm_token", op="norm", kind="int8", M=1, K=4096, pad=0, y=False),
        # a decode batch in front of an FP8 projection
        dict(name="norm_batch", op="norm", kind="e4m3", M=64, K=4096, pad=0, y=False),
        # an odd chunk of a prompt in wider buffers, the normalised rows kept for a router as well
        dict(name="norm_ragged", op="norm", kind="int8", M=1000, K=2064, pad=64, y=True),
        # a long prompt in front of a projection on 32-element blocks
        dict(name="norm_prompt", op="norm", kind="mx", M=8192, K=4096, pad=0, y=False),
        # one new token of one sequence: latency
        dict(name="rotate_token", op="rotate", code="int8", B=1, n=1, L=1000, H=8, R=4, D=128, P=64, rot=128, pairs=False),
        # one new token for each of 64 running sequences
        dict(name="rotate_decode", op="rotate", code="e4m3", B=64, n=1, L=1000, H=8, R=4, D=128, P=64, rot=128, pairs=False),
        # four drafted tokens of one very long sequence, a part of each head turned in neighbouring pairs
        dict(name="rotate_far", op="rotate", code="e4m3", B=1, n=4, L=131072, H=1, R=16, D=256, P=128, rot=64, pairs=True),
        # three prompts of different lengths written at once, one behind a cached prefix
        dict(name="rotate_prompt", op="rotate", code="int8", B=3, n=2000, L=2500, H=8, R=4, D=128, P=32, rot=128, pairs=False),
        # eight answers to one question, a token of each: latency
        dict(name="shared_answers", op="shared", code="e4m3", B=8, G=1, n=1, S=1000, O=50, H=8, R=4, D=128, P=16, causal=True),
        # a decode batch behind one system prompt
        dict(name="shared_batch", op="shared", code="int8", B=64, G=1, n=1, S=8192, O=500, H=8, R=4, D=128, P=64, causal=True),
        # a few long documents, several questions to each, four drafted tokens at once, one head of keys
        dict(name="shared_documents", op="shared", code="e4m3", B=24, G=4, n=4, S=32768, O=300, H=1, R=16, D=256, P=128, causal=True),
        # a large batch behind a long prompt, as long answers run on: reading and arithmetic
        dict(name="shared_large", op="shared", code="e4m3", B=256, G=1, n=1, S=32768, O=1500, H=8, R=4, D=128, P=64, causal=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "rotate", "shared"))
    if op == "norm":
        kind = rng.choice(("int8", "e4m3", "mx"))
        unit = {"int8": 16, "e4m3": 128, "mx": 32}[kind]
        K = unit * _spread(rng, 1, 16384 // unit)
        return dict(op=op, kind=kind, M=_spread(rng, 1, min(8192, 6144 * 4096 // K)), K=K, pad=rng.choice((0, 16, 64)),
                    y=rng.random() < 0.3)
    code, D = rng.choice(("e4m3", "int8")), rng.choice((64, 128, 256))
    P, H = rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 3, 4, 8))
    if op == "rotate":
        B, R = _spread(rng, 1, 128), rng.choice((1, 2, 4, 5, 8))
        n = _spread(rng, 1, max(2, 6000 * 1024 // (B * H * D)))
        before = _spread(rng, 1, max(2, min(2000, 40_000_000 // (B * H * D))))
        return dict(op=op, code=code, B=B, n=n, L=n + before, H=H, R=R, D=D, P=P, rot=rng.choice((D, D, D // 2, 32)),
                    pairs=rng.random() < 0.4)
    B, R, n = _spread(rng, 2, 256), rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((1, 1, 1, 2, 4, 9))
    G = min(_spread(rng, 1, 8), max(1, B // 2))
    n = max(1, min(n, 256 * 32 // (B * H * R)))
    O = max(n, _spread(rng, 1, max(2, min(4000, 250 * 1024 * 1024 // (B * H * D)))))
    S = _spread(rng, P, max(P + 1, min(65536, 128 * 32768 * 1024 // (B * n * H * R * D), 32768 * 1024 // (G * H * D))))
    return dict(op=op, code=code, B=B, G=G, n=n, S=S, O=O, H=H, R=R, D=D, P=P, causal=rng.random() < 0.8)


def _lengths(case):
    """New rows and whole length of each sequence: the first has both at their largest, the others less."""
    B, n, L = case["B"], case["n"], case["L"]
    new, whole = [], []
    for b in range(B):
        new.append(n if b == 0 else max(1, n - (n * (7 * b % 16)) // 20))
        whole.append(L if b == 0 else max(new[b], L - (L * (5 * b % 32)) // 34))
    return new, whole


def _sharing(case):
    """Group of each sequence, tokens that each group shares, new rows and own tokens of each sequence."""
    B, G, n, O, P = case["B"], case["G"], case["n"], case["O"], case["P"]
    size = [2 + 5 * g % 7 for g in range(G)]
    ends = [round(B * sum(size[: g + 1]) / sum(size)) for g in range(G)]
    group = [sum(b >= e for e in ends) for b in range(B)]
    shared = [P * max(1, (case["S"] - case["S"] * (3 * g % 8) // 10) // P) for g in range(G)]
    new = [n if b == 0 else max(1, n - (n * (7 * b % 16)) // 20) for b in range(B)]
    after = [O if b == 0 else max(new[b], O - (O * (5 * b % 32)) // 34) for b in range(B)]
    return group, shared, new, after


def _pairs(case):
    """Keys that the rows of all sequences see, in all."""
    group, shared, new, after = _sharing(case)
    seen = 0
    for g, n, o in zip(group, new, after):
        seen += n * (shared[g] + o) - (n * (n - 1) // 2 if case["causal"] else 0)
    return seen


def work(case):
    if case["op"] == "norm":
        n, scales = case["M"] * case["K"], 4 * case["M"] if case["kind"] == "int8" else case["M"] * case["K"] // BLOCK[case["kind"]]
        return {"bytes": n * (2 + 2 + 2 + 1 + 2 * case["y"]) + scales + 2 * case["K"], "flops": 0}
    row = case["H"] * case["D"]
    if case["op"] == "rotate":
        rows = sum(_lengths(case)[0])
        return {"bytes": rows * (row * (4 + 2 + 4 * case["R"]) + 4 * case["rot"]), "flops": 0}
    group, shared, new, after = _sharing(case)
    keys = sum(shared[g] for g in set(group)) + sum(after)
    return {"bytes": 2 * keys * row + 4 * sum(new) * row * case["R"], "flops": 4 * _pairs(case) * row * case["R"]}


# ---- the formats, in torch -------------------------------------------------------------------------


def _exponent(a, code):
    """The smallest e with 2^e >= a / (the format's largest magnitude), at least -127."""
    m, k = torch.frexp(a)
    top, shift = TOP[code]
    e = k - shift + (m > top).to(k.dtype)
    return torch.where(a > 0, e, torch.full_like(e, -127)).clamp_(min=-127)


def _pack_bytes(byte):
    """Scale bytes [M, blocks] -> int32 words [1, ceil(blocks / 4), 4 ceil(M / 4)]."""
    M, h = byte.shape
    full = torch.zeros((-(-M // 4) * 4, -(-h // 4) * 4), dtype=torch.uint8, device=byte.device)
    full[:M, :h] = byte
    return full.view(full.shape[0], -1, 4).permute(1, 0, 2).contiguous().view(torch.int32).view(1, -1, full.shape[0])


def _as_values(codes):
    """8-bit codes as the numbers they stand for: int8 numbers or E4M3 values."""
    return codes if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn)


def _as_scales(byte):
    return byte.view(torch.float8_e8m0fnu)


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
    # keys have a few large channels, as turned keys do
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


def _ints(values, dtype):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _offsets(new):
    return _ints([0] + np.cumsum(new).tolist(), torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        M, K, pad = case["M"], case["K"], case["pad"]
        # a residual stream has a few large channels; what a layer adds to it is smaller
        channel = 1 + 20 * (torch.rand((K,), generator=gen, device=DEV) < 0.005)
        x = torch.zeros((M, K + pad), dtype=torch.bfloat16, device=DEV)
        r = torch.zeros((M, K + pad), dtype=torch.bfloat16, device=DEV)
        x[:, :K] = 0.5 * _normal(gen, M, K)
        r[:, :K] = _normal(gen, M, K) * torch.exp(0.5 * _normal(gen, M, 1)) * channel
        s.update(x=x[:, :K], residual=r[:, :K], gamma=(1 + 0.2 * _normal(gen, K)).bfloat16())
        return s
    if case["op"] == "rotate":
        _prepare_rotate(s, case, gen)
    else:
        _prepare_shared(s, case, gen)
    return s


def _prepare_rotate(s, case, gen):
    new, whole = _lengths(case)
    H, D, P = case["H"], case["D"], case["P"]
    need = [-(-w // P) for w in whole]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((case["B"], max(need)), dtype=torch.int32, device=DEV)
    for b, at in enumerate(np.cumsum([0] + need[:-1]).tolist()):
        table[b, : need[b]] = order[at : at + need[b]]
    s["k"], s["v"], s["ks"], s["vs"] = _cache(gen, case, pages)
    s.update(table=table, offsets=_offsets(new), lens=_ints(whole, torch.int32), new=new, whole=whole)
    rows = sum(new)
    # some rows are larger than what their page holds: its scale has to grow
    loud = torch.exp2(torch.randint(-1, 3, (rows, 1, 1), generator=gen, device=DEV).float())
    s["kn"], s["vn"] = ((_normal(gen, rows, H, D) * loud).bfloat16() for _ in range(2))
    s["q"] = _normal(gen, rows, H * case["R"], D).bfloat16()
    # the pages that the new rows fall in: the scheduler that gave them out knows them
    s["touched"] = torch.cat([table[b, (w - n) // P : -(-w // P)] for b, (n, w) in enumerate(zip(new, whole))]).long()
    # cosines and sines of every position, made once
    half = case["rot"] // 2
    turn = torch.arange(max(whole), device=DEV).double()[:, None] * torch.pow(10000.0, -torch.arange(half, device=DEV).double() / half)
    s["angles"] = torch.stack((turn.cos(), turn.sin()), 1).float()


def _prepare_shared(s, case, gen):
    group, shared, new, after = _sharing(case)
    B, P = case["B"], case["P"]
    first = [shared[g] // P for g in group]
    used = sorted(set(group))
    counts = [shared[g] // P for g in used] + [-(-a // P) for a in after]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = np.cumsum([0] + counts).tolist()
    table = torch.zeros((B, max(f + c for f, c in zip(first, counts[len(used) :]))), dtype=torch.int32, device=DEV)
    for b, g in enumerate(group):
        i, j = used.index(g), len(used) + b
        table[b, : first[b]] = order[at[i] : at[i + 1]]
        table[b, first[b] : first[b] + counts[j]] = order[at[j] : at[j + 1]]
    s["k"], s["v"], s["ks"], s["vs"] = _cache(gen, case, pages)
    whole = [shared[g] + a for g, a in zip(group, after)]
    s.update(table=table, offsets=_offsets(new), lens=_ints(whole, torch.int32), group=_ints(group, torch.int32),
             shared=_ints([shared[g] for g in group], torch.int32), new=new, whole=whole)
    s["q"] = _normal(gen, sum(new), case["H"] * case["R"], case["D"]).bfloat16()
    # as a scheduler knows them: the first sequence of each group, and the longest of everything
    rows = [sum(n for n, h in zip(new, group) if h == g) for g in used]
    s["leaders"] = _ints([group.index(g) for g in used], torch.int64)
    s["dense"] = _ints([used.index(g) for g in group], torch.int64)
    s["most"] = (max(new), max(after), max(shared[g] for g in used), max(rows))


# ---- one pass -------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if op == "norm":
        codes, scale, total, y = _own_norm(s) if own else _plain_norm(s)
        scale = scale if s["case"]["kind"] == "int8" else _as_scales(scale.view(torch.uint8))
        return {"codes": _as_values(codes), "scale": scale, "sum": total, **({"y": y} if s["case"]["y"] else {})}
    if op == "rotate":
        q = _own_rotate(s) if own else _plain_rotate(s)
        return {"k": _as_values(s["k"]), "v": _as_values(s["v"]), "k_scale": _as_scales(s["ks"]), "v_scale": _as_scales(s["vs"]), "q": q}
    out, lse = _own_shared(s) if own else _plain_shared(s)
    return {"out": out, "lse": lse}


def _own_norm(s):
    import fp8_dynamic_quant_amd as wq

    case = s["case"]
    payload = {"int8": wq.WQ_PAYLOAD_INT8, "e4m3": wq.WQ_PAYLOAD_FP8_E4M3, "mx": wq.WQ_PAYLOAD_MXFP8}[case["kind"]]
    out = wq.wq_add_rms_quant(s["x"], s["residual"], s["gamma"], payload=payload, return_y=case["y"])
    return out if case["y"] else (*out, None)


def _own_rotate(s):
    import fp8_dynamic_quant_amd as wq

    cache = wq.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    return wq.wq_kv_append_rotated(cache, s["kn"], s["vn"], s["offsets"], s["lens"], s["table"], s["angles"], q=s["q"],
                                   interleaved=s["case"]["pairs"])


def _own_shared(s):
    import fp8_dynamic_quant_amd as wq

    cache = wq.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    return wq.wq_kv_attention_shared(cache, s["q"], s["offsets"], s["lens"], s["table"], s["group"], s["shared"],
                                     causal=s["case"]["causal"], return_lse=True)


def _plain_norm(s):
    kind, K = s["case"]["kind"], s["case"]["K"]
    total = (s["x"].float() + s["residual"].float()).bfloat16()
    h = total.float()
    # the sum of squares and what stands next to a rounding border in 64 bits, each rounded once to 32
    mean = (h.double().square().sum(-1, keepdim=True) / K).float() + 1e-6
    inv = (1 / mean.double().sqrt().float().double()).float()
    v = h * inv * s["gamma"].float()
    y = v.bfloat16() if s["case"]["y"] else None
    if kind == "int8":
        scale = (v.abs().amax(-1).double() / 127).float()
        codes = torch.round((v.double() / scale.double()[:, None]).float())
        return torch.where(scale[:, None] > 0, codes, torch.zeros_like(codes)).to(torch.int8), scale, total, y
    blocks = v.view(v.shape[0], -1, BLOCK[kind])
    e = _exponent(blocks.abs().amax(-1), "e4m3")
    codes = torch.ldexp(blocks, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(-1, 1, K), _pack_bytes((e + 127).to(torch.uint8)), total, y


def _row_places(s):
    """Sequence, index among its new rows and position of every row."""
    r = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(s["offsets"], r, right=True) - 1
    i = r - s["offsets"][b]
    n = s["offsets"][b + 1] - s["offsets"][b]
    return b, i, s["lens"][b] - n + i


def _turned(x, angles, at, case):
    """f32 rows [T, heads, D], their first rot elements turned by the angles of their positions."""
    rot, half = case["rot"], case["rot"] // 2
    c, d = angles[at].unsqueeze(1).unbind(2)
    out = x.clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["pairs"] else (slice(0, half), slice(half, rot))
    out[..., one] = x[..., one] * c - x[..., two] * d
    out[..., two] = x[..., two] * c + x[..., one] * d
    return out


def _plain_rotate(s):
    case = s["case"]
    code, P = case["code"], case["P"]
    b, _, at = _row_places(s)
    page, slot = s["table"][b, at // P].long(), at % P
    touched = s["touched"]
    # the first new slot of every page: what stands before it is kept, at the page's new scale
    first = torch.full((s["ks"].shape[0],), P, device=DEV).scatter_reduce_(0, page, slot, "amin")[touched]
    kept, before = first[:, None] > 0, (torch.arange(P, device=DEV) < first[:, None])[:, None]

    def put(codes, scale, x, columns):
        most = torch.zeros(scale.shape, device=DEV)
        most.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
        new, old = _exponent(most[touched], code), scale[touched].int() - 127
        e = torch.where(kept, torch.maximum(old, new), new)
        shift = torch.where(kept, old - e, torch.zeros_like(e))
        scale[touched] = (e + 127).to(torch.uint8)
        y = torch.ldexp(x, 127 - scale[page].int()[..., None])
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

    put(s["k"], s["ks"], _turned(s["kn"].float(), s["angles"], at, case), False)
    put(s["v"], s["vs"], s["vn"].float(), True)
    return _turned(s["q"].float(), s["angles"], at, case).bfloat16()


def _plain_shared(s):
    """Each group's rows over the pages that it shares, each sequence's over its own, then both sums as one."""
    case = s["case"]
    B, H, R, D, P = case["B"], case["H"], case["R"], case["D"], case["P"]
    most_new, most_own, most_shared, most_rows = s["most"]
    b, i, _ = _row_places(s)
    table, first = s["table"].long(), s["shared"].long() // P
    x = s["q"].float().view(-1, H, R, D)

    def gather(codes, scale, pages):
        v = codes[pages] if codes.dtype == torch.int8 else codes.view(torch.float8_e4m3fn)[pages]
        return v.float() * torch.ldexp(torch.ones((), device=DEV), scale[pages].int() - 127)[..., None, None]

    def over(q, pages, see, most):
        """q [N, H, rows, D] over the pages [N, width]: maximum, sum and weighted values of what the rows see."""
        n = q.shape[0]
        k = gather(s["k"], s["ks"], pages).transpose(1, 2).reshape(n, H, -1, D)[:, :, :most]
        v = gather(s["v"], s["vs"], pages).permute(0, 2, 1, 4, 3).reshape(n, H, -1, D)[:, :, :most]
        score = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(D**-0.5).masked_fill_(~see, float("-inf"))
        top = score.amax(-1, keepdim=True)
        p = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
        return top, p.sum(-1, keepdim=True), torch.matmul(p, v)

    # rows by group, each group's in order
    g = s["dense"][b]
    places = torch.zeros((len(s["leaders"]), most_rows), dtype=torch.bool, device=DEV)
    counts = torch.zeros(len(s["leaders"]), dtype=torch.int64, device=DEV).scatter_add_(0, g, torch.ones_like(g))
    at = torch.arange(len(g), device=DEV) - (counts.cumsum(0) - counts)[g]
    of_group = torch.zeros((*places.shape, H, R, D), device=DEV)
    of_group[g, at] = x
    of_group = of_group.permute(0, 2, 1, 3, 4).reshape(-1, H, most_rows * R, D)
    j = torch.arange(most_shared, device=DEV)
    see = (j < s["shared"][s["leaders"]][:, None])[:, None, None]
    both = [[t.view(-1, H, most_rows, R, t.shape[-1]).permute(0, 2, 1, 3, 4)[g, at]
             for t in over(of_group, table[s["leaders"], : -(-most_shared // P)], see, most_shared)]]
    # rows by sequence
    of_own = torch.zeros((B, most_new, H, R, D), device=DEV)
    of_own[b, i] = x
    of_own = of_own.permute(0, 2, 1, 3, 4).reshape(B, H, most_new * R, D)
    j = torch.arange(most_own, device=DEV)
    count = (s["lens"].long() - s["shared"])[:, None].expand(B, most_new)
    if case["causal"]:
        count = count - (s["offsets"][1:] - s["offsets"][:-1])[:, None] + 1 + torch.arange(most_new, device=DEV)
    see = (j < count[..., None])[:, :, None].expand(B, most_new, R, most_own).reshape(B, 1, most_new * R, most_own)
    cols = first[:, None] + torch.arange(-(-most_own // P), device=DEV)
    pages = torch.gather(table, 1, cols.clamp(max=table.shape[1] - 1))
    both.append([t.view(B, H, most_new, R, t.shape[-1]).permute(0, 2, 1, 3, 4)[b, i] for t in over(of_own, pages, see, most_own)])
    (m0, l0, o0), (m1, l1, o1) = both
    top = torch.maximum(m0, m1)
    w0, w1 = (torch.exp(m - top) for m in (m0, m1))
    total = w0 * l0 + w1 * l1
    out = (w0 * o0 + w1 * o1) / total
    return out.reshape(-1, H * R, D).bfloat16(), (top + total.log()).reshape(-1, H * R)


# ---- the definition in 64 bits ---------------------------------------------------------------------


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


GRID_E4M3 = np.array([m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def _host(t):
    return t.detach().to("cpu").double().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def _decode64(codes):
    """E4M3 bytes -> f64, from the fields of a code."""
    c = codes.to(torch.int64)
    sign, ef, f = c // 128, c // 8 % 16, (c % 8).double() / 8
    v = torch.where(ef == 0, f * 2.0**-6, (1 + f) * torch.pow(2.0, (ef - 7).double()))
    return v * (1 - 2 * sign)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    return _exact_rotate(s, case) if case["op"] == "rotate" else _exact_shared(s, case)


def _exact_norm(s, case):
    M, K = case["M"], case["K"]
    total = s["x"].double() + s["residual"].double()
    # the residual stream is in bf16: what is normalised is the sum as it is handed on
    h = total.bfloat16().double()
    v = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["gamma"].double()
    out = {"codes": None, "scale": None, "sum": total, **({"y": v} if case["y"] else {})}
    if case["kind"] == "int8":
        out["scale"] = v.abs().amax(-1) / 127
        return out
    blocks = _host(v).reshape(M, -1, BLOCK[case["kind"]])
    e = _block_exponent64(np.abs(blocks).max(-1), 448.0)
    out["codes"] = torch.from_numpy(_nearest64(np.ldexp(blocks, -e[..., None]), GRID_E4M3).reshape(M, 1, K))
    byte = np.zeros((-(-M // 4) * 4, -(-e.shape[1] // 4) * 4), dtype=np.int64)
    byte[:M, : e.shape[1]] = e + 127
    words = byte.reshape(byte.shape[0], -1, 4).transpose(1, 0, 2).reshape(1, byte.shape[1] // 4, -1)
    out["scale"] = torch.from_numpy(np.ldexp(1.0, words - 127))
    return out


def _exact_turned(x, angles, at, case):
    """f64 rows [T, heads, D]: the first rot elements as complex numbers, times those of the angles."""
    rot, half = case["rot"], case["rot"] // 2
    turn = (angles[at, 0] + 1j * angles[at, 1])[:, None]
    head = x[..., :rot]
    z = head[..., 0::2] + 1j * head[..., 1::2] if case["pairs"] else head[..., :half] + 1j * head[..., half:]
    z = z * turn
    z = np.stack((z.real, z.imag), -1).reshape(head.shape) if case["pairs"] else np.concatenate((z.real, z.imag), -1)
    return np.concatenate((z, x[..., rot:]), -1)


def _exact_rotate(s, case):
    P, code = case["P"], case["code"]
    table, angles = _host(s["table"]), _host(s["angles"])
    at = np.concatenate([np.arange(w - n, w) for n, w in zip(s["new"], s["whole"])])
    rows = {"k": _exact_turned(_host(s["kn"].float()), angles, at, case), "v": _host(s["vn"].float())}
    out = {}
    for side, transposed in (("k", False), ("v", True)):
        held = s[side]
        held = _host(held.double()) if code == "int8" else _host(_decode64(held))
        held = held.swapaxes(-1, -2).copy() if transposed else held
        e = _host(s[side + "s"]).astype(np.int64) - 127
        row = 0
        for b, (n, whole) in enumerate(zip(s["new"], s["whole"])):
            for pg in range((whole - n) // P, -(-whole // P)):
                lo, hi = max(whole - n, pg * P), min(whole, (pg + 1) * P)
                part = rows[side][row : row + hi - lo].swapaxes(0, 1)  # [H, rows, D]
                row += hi - lo
                page, slot = table[b, pg], lo - pg * P
                en = _block_exponent64(np.abs(part).max((-1, -2)), 127.0 if code == "int8" else 448.0)
                if slot > 0:
                    en = np.maximum(en, e[page])
                    old = np.ldexp(held[page][:, :slot], (e[page] - en)[:, None, None])
                    held[page, :, :slot] = np.rint(old) if code == "int8" else _nearest64(old, GRID_E4M3)
                # slots behind the new rows keep their codes
                y = np.ldexp(part, -en[:, None, None])
                held[page, :, slot : slot + hi - lo] = np.rint(y) if code == "int8" else _nearest64(y, GRID_E4M3)
                e[page] = en
        held = held.swapaxes(-1, -2).copy() if transposed else held
        # codes of int8 are whole numbers, which 64 bits may round the other way: no value
        out[side] = None if code == "int8" else torch.from_numpy(held)
        out[side + "_scale"] = torch.from_numpy(np.ldexp(1.0, e))
    q = _exact_turned(_host(s["q"].float()), angles, at, case)
    return {"k": out["k"], "v": out["v"], "k_scale": out["k_scale"], "v_scale": out["v_scale"], "q": torch.from_numpy(q)}


def _exact_shared(s, case):
    H, R, D, P, code = case["H"], case["R"], case["D"], case["P"], case["code"]
    if _pairs(case) * H * R * D > 3e12:
        return None
    q, rows = s["q"].double(), s["q"].shape[0]
    out = torch.zeros((rows, H * R, D), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, H * R), -math.inf, dtype=torch.float64, device=DEV)
    group, shared, _, _ = _sharing(case)

    def of_head(side, pages, h):
        c = s[side][pages, h]
        c = c.double() if code == "int8" else _decode64(c)
        return c * torch.pow(2.0, s[side + "s"][pages, h].double() - 127)[:, None, None]

    for h in range(H):
        row, of, front = 0, None, None
        for b, (n, whole) in enumerate(zip(s["new"], s["whole"])):
            pages = s["table"][b, : -(-whole // P)].long()
            cut = shared[group[b]] // P
            if group[b] != of:  # what a group shares is decoded once
                of = group[b]
                front = of_head("k", pages[:cut], h).reshape(-1, D), of_head("v", pages[:cut], h).transpose(1, 2).reshape(-1, D)
            k = torch.cat((front[0], of_head("k", pages[cut:], h).reshape(-1, D)))[:whole]
            v = torch.cat((front[1], of_head("v", pages[cut:], h).transpose(1, 2).reshape(-1, D)))[:whole]
            z = (q[row : row + n, h * R : h * R + R].reshape(n * R, D) @ k.t().contiguous()) / math.sqrt(D)
            if case["causal"]:
                hide = torch.full((n, whole), -math.inf, dtype=torch.float64, device=DEV).triu(whole - n + 1)
                z = z + hide.repeat_interleave(R, 0)
            lse[row : row + n, h * R : h * R + R] = torch.logsumexp(z, -1).view(n, R)
            out[row : row + n, h * R : h * R + R] = (torch.softmax(z, -1) @ v).view(n, R, D)
            row += n
    return {"out": out, "lse": lse}
