"""The attention block of a decode step, measured: rotary positions, the low-bit KV cache and attention over it.

Each case is one call (or one pair of calls) of the public entry points, beside a plain form of the same operator in
elementary fp32 tensor operations and a 64-bit evaluation of its definition.  `own` chooses the entry points.

Head shapes are those of the 7B, 14B and 70B decoder layers of `synth.LAYER_SHAPES` (128-wide heads: 32 over 32,
40 over 40 and 64 over 8), with a generic 64-wide head for the narrow variant.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

GROUP = 32          # dims that share a scale and an offset
TILE = 16           # tokens of a cache tile
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- the cases ----------------------------------------------------------------------

def _table(name, rows, rot, factor):
    return dict(name=name, op="table", rows=rows, rot=rot, base=10000.0, factor=factor, original=8192, low=1.0, high=32.0,
                mscale=1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0)


def _rotate(name, n, heads, D, rot, layout, dtype, inverse, pad):
    return dict(name=name, op="rotate", n=n, heads=heads, D=D, rot=rot, layout=layout, dtype=dtype, inverse=inverse, pad=pad)


def _append(name, n, hq, hkv, D, rot, bits, layout, dtype, page):
    return dict(name=name, op="append", n=n, hq=hq, hkv=hkv, D=D, rot=rot, bits=bits, layout=layout, dtype=dtype, page=page)


def _attend(name, B, T, hq, hkv, D, bits, page, longest, shortest, prefix, dtype):
    return dict(name=name, op="attend", B=B, T=T, hq=hq, hkv=hkv, D=D, bits=bits, page=page, longest=longest,
                shortest=shortest, prefix=prefix, dtype=dtype)


def listed():
    return [
        # the rotation table of a model served at 128 Ki tokens, frequencies scaled by parts from 8 Ki
        _table("table_128k", 131072, 128, 16.0),
        # q of one 14B layer at prefill (2048 tokens), rotated whole
        _rotate("rotate_prefill", 2048, 40, 128, 128, "half", "bf16", False, 0),
        # the gradient of a rotation of part of the head, read out of a wider fused projection row
        _rotate("rotate_grad_part", 1111, 64, 64, 32, "interleaved", "f16", True, 192),
        # one decode step of 16 requests, 7B heads: q and k rotated, k and v written to a 4-bit cache, read back
        _append("append_decode", 16, 32, 32, 128, 128, 4, "half", "bf16", 64),
        # a prefill of 2048 tokens, 70B heads, 8-bit cache
        _append("append_prefill", 2048, 64, 8, 128, 128, 8, "half", "bf16", 64),
        # a ragged chunk of prompts with narrow heads, part of the head rotated, small pages
        _append("append_odd", 5003, 16, 4, 64, 32, 4, "interleaved", "f16", 16),
        # one request, a short context, 7B heads: latency
        _attend("attend_one_short", 1, 1, 32, 32, 128, 4, 64, 333, 333, 0, "bf16"),
        # one request at 128 Ki tokens, 70B heads, 4-bit cache
        _attend("attend_one_long", 1, 1, 64, 8, 128, 4, 64, 131072, 131072, 0, "bf16"),
        # a batch of ragged contexts, 14B heads, 8-bit cache
        _attend("attend_ragged", 24, 1, 40, 40, 128, 8, 32, 4001, 1, 0, "bf16"),
        # four draft tokens of each of eight requests checked at once, narrow heads, small pages
        _attend("attend_draft", 8, 4, 32, 8, 64, 4, 16, 6000, 500, 0, "f16"),
        # two requests that share a system prompt, 7B heads
        _attend("prefix_small", 2, 1, 32, 32, 128, 8, 64, 200, 50, 1000, "bf16"),
        # 48 requests over one long shared document, 70B heads
        _attend("prefix_large", 48, 1, 64, 8, 128, 4, 64, 700, 1, 32100, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rotate", "append", "attend", "attend", "prefix"])
    layout, dtype = rng.choice(["half", "interleaved"]), rng.choice(["bf16", "bf16", "f16"])
    bits, page, D = rng.choice([4, 8]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    hq, hkv = rng.choice([(32, 32), (40, 40), (64, 8), (32, 8), (16, 4), (24, 2)])
    if op == "table":
        c = _table("", _log(rng, 1000, 131072), rng.choice([32, 64, 128]), rng.choice([1.0, 4.0, 16.0]))
    elif op == "rotate":
        c = _rotate("", _log(rng, 1, 2048), hq, D, rng.choice([D, D, D // 2, 32]), layout,
                    rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5, rng.choice([0, 0, 64, 4]))
    elif op == "append":
        c = _append("", _log(rng, 1, 2048), hq, hkv, D, rng.choice([D, D, D // 2]), bits, layout, dtype, page)
    elif op == "attend":
        hkv = min(hkv, 16)
        hq = hkv * rng.choice([1, 4, 8])
        B, T = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 5])
        longest = _log(rng, 16, max(17, min(131072, 130_000_000 // (B * hkv * D))))
        c = _attend("", B, T, hq, hkv, D, bits, page, longest, rng.choice([1, longest // 2 + 1, longest]), 0, dtype)
    else:
        hkv = min(hkv, 8)
        hq = hkv * rng.choice([1, 4, 8])
        B, T = _log(rng, 2, 48), rng.choice([1, 1, 2])
        c = _attend("", B, T, hq, hkv, D, bits, page, _log(rng, 1, 700), 1, _log(rng, 200, 32100 // T), dtype)
    del c["name"]
    return c


# ---- what a user has in hand --------------------------------------------------------

def _tile_bytes(D, bits):
    return TILE * (2 * D * bits // 8 + 2 * (D // GROUP) * 4)


def _lens(case, seed):
    g = torch.Generator().manual_seed(int(seed) * 7 + 1)
    n = torch.randint(case["shortest"], case["longest"] + 1, (case["B"],), generator=g, dtype=torch.int32)
    n[0] = case["longest"]
    return n


def _frequencies(case):
    """Rotation frequencies (radians per position) of a table case, in 64 bits."""
    f = [case["base"] ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
    out = []
    for x in f:
        turns = case["original"] * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - case["low"]) / (case["high"] - case["low"])))
        out.append(x * (keep + (1.0 - keep) / case["factor"]))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "table":
        # (the seed moves the window of positions: a table is a function of its sizes alone)
        st["first"] = int(seed) % 9973
        return st
    if case["op"] in ("rotate", "append"):
        n, rows = case["n"], 4096
        # ordinary rows of cos | sin, at positions that jump as those of several requests do
        p = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None]
        f = 10000.0 ** (-2.0 * torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) / case["rot"])
        st["table"] = torch.cat([torch.cos(p * f), torch.sin(p * f)], 1).float()
        st["positions"] = torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "rotate":
        wide = randn(n, case["heads"] * case["D"] + case["pad"]).to(DT[case["dtype"]])
        st["x"] = wide[:, case["pad"]:].unflatten(1, (case["heads"], case["D"]))
        return st
    D, bits, page, hkv = case["D"], case["bits"], case["page"], case["hkv"]
    tb = _tile_bytes(D, bits)
    if case["op"] == "append":
        row = randn(n, case["hq"] + 2 * hkv, D)
        # keys have channels that stand far out, as rotated keys do
        row[:, case["hq"]:case["hq"] + hkv, :: 37] *= 6.0
        row = row.to(DT[case["dtype"]])             # one fused q | k | v projection row per token
        st["q"], st["k"], st["v"] = row.split([case["hq"], hkv, hkv], 1)
        pages = -(-n // page) + 3
        st["pages"] = torch.zeros((pages, hkv, page // TILE, tb), dtype=torch.uint8, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(n, device="cuda") + int(seed) % (2 * page)
        st["slots"] = order[at // page] * page + at % page
        return st
    B, prefix = case["B"], case["prefix"]
    lens = _lens(case, seed)
    each = -(-case["longest"] // page)
    shared = -(-prefix // page)
    pages = B * each + shared
    t = torch.randint(0, 256, (pages, hkv, page // TILE, tb), generator=g, device="cuda", dtype=torch.uint8)
    # scales and offsets of groups that spread about zero, a few of the key groups six times as wide
    G, kb = D // GROUP, TILE * D * bits // 8
    top = 2.0 ** bits - 1
    shape = (pages, hkv, page // TILE, TILE, G)
    s = (torch.rand(shape, generator=g, device="cuda") + 3.5) / top
    wide = (torch.rand((1, hkv, 1, 1, G), generator=g, device="cuda") < 0.1).float() * 5.0 + 1.0
    ks = (s * wide).half()
    kz = (-0.5 * top * ks.float() + 0.3 * randn(*shape)).half()
    vs = ((torch.rand(shape, generator=g, device="cuda") + 3.5) / top).half().transpose(3, 4).contiguous()
    vz = (-0.5 * top * vs.float() + 0.3 * randn(*vs.shape)).half()
    for i, m in enumerate((ks, kz, vs, vz)):
        o = 2 * kb + 2 * TILE * G * i
        t[..., o:o + 2 * TILE * G] = m.reshape(*shape[:3], -1).view(torch.uint8)
    st["pages"] = t
    order = torch.randperm(pages, generator=g, device="cuda").int()
    st["block_table"], st["prefix_table"] = order[:B * each].view(B, each), order[B * each:]
    st["lens"] = lens.cuda()
    st["q"] = randn(B, case["T"], case["hq"], D).to(DT[case["dtype"]])
    return st


# ---- one pass -----------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _handle():
    import bit_weight_quantized_dequant_gb300 as lq
    return lq, lq.Handle(0)


def _cache(st):
    if "cache" not in st:      # a descriptor of the pages, which a program keeps beside them
        lq, _ = _handle()
        c = st["case"]
        st["cache"] = lq.KVCache(st["pages"], page_size=c["page"], kv_heads=c["hkv"], head_dim=c["D"], bits=c["bits"])
    return st["cache"]


def _run_own(st):
    lq, h = _handle()
    c = st["case"]
    if c["op"] == "table":
        return h.rope_table(c["rows"], c["rot"], base=c["base"], first=st["first"], factor=c["factor"],
                            original_length=c["original"], low_rotations=c["low"], high_rotations=c["high"],
                            mscale=c["mscale"])
    if c["op"] == "attend":
        return h.kv_attention(st["q"], _cache(st), st["block_table"], st["lens"], scale=c["D"] ** -0.5,
                              prefix_table=st["prefix_table"] if c["prefix"] else None, prefix_len=c["prefix"])
    layout = lq.ROPE_HALF if c["layout"] == "half" else lq.ROPE_INTERLEAVED
    if c["op"] == "rotate":
        return h.rope(st["x"], st["positions"], st["table"], layout=layout, inverse=c["inverse"])
    q = h.kv_append(_cache(st), st["k"], st["v"], st["slots"], q=st["q"], table=st["table"], positions=st["positions"],
                    layout=layout)
    k, v = h.kv_read(_cache(st), st["slots"], dtype=DT[c["dtype"]])
    return [q, k, v]


def run(st):
    if own:
        return _run_own(st)
    return {"table": _plain_table, "rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[st["case"]["op"]](st)


# ---- the plain forms ----------------------------------------------------------------

def _plain_table(st):
    c = st["case"]
    # frequencies in turns as 64-bit fractions: the product with a position wraps modulo one turn, exactly
    u = torch.tensor([round(f / (2 * math.pi) * 2 ** 64) for f in _frequencies(c)], dtype=torch.int64, device="cuda")
    p = torch.arange(st["first"], st["first"] + c["rows"], device="cuda", dtype=torch.int64)
    a = (p[:, None] * u).float() * (2 * math.pi * 2.0 ** -64)
    return torch.cat([torch.cos(a) * c["mscale"], torch.sin(a) * c["mscale"]], 1)


def _rotated(x, st, inverse):
    """x [n][heads][D], in 32 bits."""
    c = st["case"]
    rot, x = c["rot"], x.float()
    cs = st["table"][st["positions"].long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    part, rest = x[..., :rot], x[..., rot:]
    if c["layout"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    else:
        a, b = part[..., 0::2], part[..., 1::2]
    if inverse:
        pa, pb = a * cos + b * sin, b * cos - a * sin
    else:
        pa, pb = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([pa, pb], -1) if c["layout"] == "half" else torch.stack([pa, pb], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_rotate(st):
    return _rotated(st["x"], st, st["case"]["inverse"]).to(st["x"].dtype)


def _through_cache(x, bits):
    """x [..., D] as a group-of-32 low-bit cache holds it, in 32 bits."""
    top = float(2 ** bits - 1)
    y = x.float().clamp(-65504.0, 65504.0).unflatten(-1, (-1, GROUP))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    z, s = lo.half().float(), ((hi - lo) * (1.0 / top)).half().float()
    code = torch.where(s > 0, torch.round((y - z) / s).clamp(0.0, top), torch.zeros_like(y))
    return (code * s + z).flatten(-2)


def _plain_append(st):
    c = st["case"]
    q, k = (_rotated(st[n], st, False).to(st[n].dtype) for n in ("q", "k"))
    return [q, _through_cache(k, c["bits"]).to(k.dtype), _through_cache(st["v"], c["bits"]).to(k.dtype)]


def _unpacked(t, D, bits):
    """Tiles [..., bytes] -> keys and values [..., 16, D] in 32 bits."""
    G, kb, per = D // GROUP, TILE * D * bits // 8, 32 // bits
    lead = t.shape[:-1]
    shift = torch.arange(0, 32, bits, device=t.device, dtype=torch.int32)

    def codes(o):      # [..., row (8), column (4), word of the lane, code of the word]
        w = t[..., o:o + kb].view(torch.int32).view(*lead, -1, 32, 4).transpose(-3, -2).reshape(*lead, 8, 4, -1)
        return (w[..., None] >> shift) & (2 ** bits - 1)

    def meta(i, *shape):
        o = 2 * kb + 2 * TILE * G * i
        return t[..., o:o + 2 * TILE * G].view(torch.float16).view(*lead, *shape).float()

    d = len(lead)
    at = lambda *order: tuple(range(d)) + tuple(d + o for o in order)  # noqa: E731
    k = codes(0).view(*lead, 8, 4, 2, G, 8 // per, per).permute(at(2, 0, 3, 1, 4, 5)).reshape(*lead, TILE, G, GROUP)
    k = k * meta(0, TILE, G)[..., None] + meta(1, TILE, G)[..., None]
    W = D // 8 // per
    v = codes(kb).view(*lead, 8, 4, 2, 2, W, per).permute(at(2, 1, 3, 5, 4, 0)).reshape(*lead, TILE, G, GROUP)
    s, z = (meta(i, G, 4, 2, 2).permute(at(2, 1, 3, 0)).reshape(*lead, TILE, G, 1) for i in (2, 3))
    return k.flatten(-2), (v * s + z).flatten(-2)


def _plain_attend(st):
    c = st["case"]
    B, T, hq, hkv, D, P = c["B"], c["T"], c["hq"], c["hkv"], c["D"], c["prefix"]
    q = st["q"].float().view(B, T, hkv, hq // hkv, D) * D ** -0.5

    def held(table):   # pages [..., m] -> keys and values [..., hkv, tokens, D]
        return [x.movedim(-4, -5).flatten(-4, -2) for x in _unpacked(st["pages"][table.long()], D, c["bits"])]

    k, v = held(st["block_table"])
    at = torch.arange(k.shape[2], device=k.device)
    seen = st["lens"][:, None, None] - T + 1 + torch.arange(T, device=k.device)[:, None]       # [B, T, 1]
    mask = (at < seen)[:, :, None, None]
    score = torch.einsum("bthgd,bhnd->bthgn", q, k).masked_fill(~mask, -math.inf)
    v = torch.where((at < st["lens"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    top = score.amax(-1, keepdim=True)
    if P:
        pk, pv = (x[:, :P] for x in held(st["prefix_table"]))
        before = torch.einsum("bthgd,hnd->bthgn", q, pk)
        top = torch.maximum(top, before.amax(-1, keepdim=True))
    safe = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - safe)
    total, o = p.sum(-1, keepdim=True), torch.einsum("bthgn,bhnd->bthgd", p, v)
    if P:
        p = torch.exp(before - safe)
        total, o = total + p.sum(-1, keepdim=True), o + torch.einsum("bthgn,hnd->bthgd", p, pv)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return [o.view(B, T, hq, D).to(st["q"].dtype), (safe + torch.log(total)).view(B, T, hq)]


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    c = case
    if c["op"] == "table":
        return {"bytes": 4.0 * c["rows"] * c["rot"], "flops": 4.0 * c["rows"] * c["rot"]}
    e = DT[c["dtype"]].itemsize
    if c["op"] == "rotate":
        return {"bytes": c["n"] * (2.0 * c["heads"] * c["D"] * e + 4 * c["rot"]), "flops": 3.0 * c["n"] * c["heads"] * c["rot"]}
    held = c["hkv"] * _tile_bytes(c["D"], c["bits"]) / TILE          # bytes a token holds in the cache
    if c["op"] == "append":
        # q, k, v and the table rows in, q and the cache out; the cache in, k and v out
        b = c["n"] * ((2 * c["hq"] + 4 * c["hkv"]) * c["D"] * e + 4 * c["rot"] + 2 * held)
        return {"bytes": float(b), "flops": 10.0 * c["n"] * (c["hq"] + 2 * c["hkv"]) * c["D"]}
    # lengths are drawn evenly from shortest to longest, the first is the longest
    kept = c["longest"] + (c["B"] - 1) * 0.5 * (c["shortest"] + c["longest"])
    rows = c["B"] * c["T"] * c["hq"]
    b = held * (kept + c["prefix"]) + rows * (2.0 * c["D"] * e + 4)
    return {"bytes": float(b), "flops": 4.0 * c["D"] * c["T"] * c["hq"] * (kept + c["B"] * c["prefix"])}


# ---- the definitions in 64 bits -----------------------------------------------------

def _turn64(x, st, inverse):
    c = st["case"]
    rot, y = c["rot"], x.double().clone()
    sign = -1.0 if inverse else 1.0
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        cs = st["table"][st["positions"].long()].double()
        co, si = cs[:, i, None], sign * cs[:, rot // 2 + i, None]
        u, w = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * co - w * si, u * si + w * co
    return y


def _held64(x, bits):
    y = x.double().clamp(-65504.0, 65504.0).reshape(*x.shape[:-1], -1, GROUP)
    z = y.min(-1, keepdim=True).values.half().double()
    s = ((y.max(-1, keepdim=True).values - y.min(-1, keepdim=True).values) / (2 ** bits - 1)).half().double()
    c = torch.round((y - z) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 2 ** bits - 1)
    return (torch.where(s > 0, c, torch.zeros_like(c)) * s + z).reshape(x.shape)


def _values64(tiles, D, bits):
    """Tiles [m, bytes] -> keys and values [m * 16, D] in 64 bits, each value fetched from where it lies."""
    G, kb, per = D // GROUP, TILE * D * bits // 8, 32 // bits
    tok = torch.arange(TILE, device="cuda")[:, None]
    dim = torch.arange(D, device="cuda")[None]

    def code(lane, word, e, o):
        byte = o + (word // 4) * 512 + lane * 16 + (word % 4) * 4 + e * bits // 8
        return ((tiles[:, byte].int() >> (e * bits % 8)) & (2 ** bits - 1)).double()

    def half(i, at):
        return tiles[:, 2 * kb + 2 * TILE * G * i:2 * kb + 2 * TILE * G * (i + 1)].contiguous().view(torch.float16)[:, at].double()

    g, r = dim // GROUP, dim % GROUP
    per_group = 8 // per                                    # key words of a lane in one group
    word = (tok // 8) * (G * per_group) + g * per_group + (r % 8) // per
    k = code(4 * (tok % 8) + r // 8, word, r % per, 0) * half(0, tok * G + g) + half(1, tok * G + g)
    W = D // 8 // per
    slab, n = dim // 8, dim % 8
    j = (tok & 1) + 2 * (tok // 8)
    at = g * TILE + 4 * ((tok % 8) // 2) + (tok & 1) + 2 * (tok // 8)
    v = code(4 * n + (tok % 8) // 2, j * W + slab % W, slab // W, kb) * half(2, at) + half(3, at)
    return k.reshape(-1, D), v.reshape(-1, D)


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "table":
        p = torch.arange(st["first"], st["first"] + c["rows"], device="cuda", dtype=torch.float64)[:, None]
        a = p * torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
        return torch.cat([torch.cos(a), torch.sin(a)], 1) * c["mscale"]
    if c["op"] == "rotate":
        return _turn64(st["x"], st, c["inverse"])
    if c["op"] == "append":
        q, k = _turn64(st["q"], st, False), _turn64(st["k"], st, False).to(DT[c["dtype"]])
        return [q, _held64(k, c["bits"]), _held64(st["v"], c["bits"])]
    B, T, hq, hkv, D, P = c["B"], c["T"], c["hq"], c["hkv"], c["D"], c["prefix"]
    if B * c["longest"] * hkv * D > 1 << 31:
        return None
    out = torch.zeros((B, T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, hq), dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    for h in range(hkv):
        shared = _values64(st["pages"][st["prefix_table"].long(), h].flatten(0, 1), D, c["bits"]) if P else None
        for b in range(B):
            used = st["block_table"][b, :max(1, -(-lens[b] // c["page"]))].long()
            k, v = (x[:lens[b]] for x in _values64(st["pages"][used, h].flatten(0, 1), D, c["bits"]))
            if P:
                k, v = torch.cat([shared[0][:P], k]), torch.cat([shared[1][:P], v])
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for t in range(T):
                n = P + max(0, lens[b] - T + 1 + t)
                s = (st["q"][b, t, heads].double() @ k[:n].T) * D ** -0.5
                lse[b, t, heads] = torch.logsumexp(s, -1)
                out[b, t, heads] = torch.softmax(s, -1) @ v[:n]
    return [out, lse]
