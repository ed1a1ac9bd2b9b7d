"""Long prompts over the low-bit KV cache, measured: attention of chunks of new tokens, attention through a sliding
window with sinks, and the log probabilities that a scored prompt or a decode step ends in.

Each case is one call (or a call and its gradient) of the public entry points, beside a plain form of the same operator
in elementary tensor operations and a 64-bit evaluation of its definition.  `own` chooses the entry points.

Head shapes are those of the 7B, 14B and 70B decoder layers of `synth.LAYER_SHAPES` (128-wide heads: 32 over 32, 40 over
40 and 64 over 8), with a generic 64-wide head for the narrow variant; vocabularies are generic.
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

def _chunk(name, B, new, past, hq, hkv, D, bits, page, dtype, window=0, sinks=0):
    """B requests of 1 to `new` new tokens each (the first: `new`), after 0 to `past` earlier ones (the first: `past`)."""
    return dict(name=name, op="chunk", B=B, new=new, past=past, hq=hq, hkv=hkv, D=D, bits=bits, page=page, dtype=dtype,
                window=window, sinks=sinks)


def _decode(name, B, T, longest, shortest, hq, hkv, D, bits, page, dtype, window, sinks):
    return dict(name=name, op="decode", B=B, T=T, longest=longest, shortest=shortest, hq=hq, hkv=hkv, D=D, bits=bits,
                page=page, dtype=dtype, window=window, sinks=sinks)


def _score(name, n, V, dtype, top, grad=False, pad=0, ignored=0.0, banned=0.0):
    return dict(name=name, op="score", n=n, V=V, dtype=dtype, top=top, grad=grad, pad=pad, ignored=ignored, banned=banned)


def listed():
    return [
        # the last piece of one short prompt, 7B heads, 4-bit cache: latency
        _chunk("chunk_short", 1, 65, 300, 32, 32, 128, 4, 64, "bf16"),
        # a whole prompt of 2048 tokens at once, 14B heads, 8-bit cache
        _chunk("chunk_prompt", 1, 2048, 0, 40, 40, 128, 8, 64, "bf16"),
        # twelve requests at different places of their prompts in one call, 7B heads, small pages
        _chunk("chunk_ragged", 12, 701, 6001, 32, 32, 128, 4, 32, "bf16"),
        # the last 2048 tokens of a prompt of 32 Ki, 70B heads, 4-bit cache
        _chunk("chunk_long", 1, 2048, 30720, 64, 8, 128, 4, 64, "bf16"),
        # chunks through a window with sinks, narrow heads, an odd window, small pages
        _chunk("chunk_window", 3, 1111, 8003, 16, 4, 64, 8, 16, "f16", 1001, 5),
        # one request at 128 Ki tokens that sees its last 4096 and the first four, 70B heads
        _decode("window_one", 1, 1, 131072, 131072, 64, 8, 128, 4, 64, "bf16", 4096, 4),
        # a batch of ragged contexts through a window, 14B heads, 8-bit cache
        _decode("window_batch", 32, 1, 5001, 100, 40, 40, 128, 8, 32, "bf16", 1024, 16),
        # four draft tokens of each of eight requests, narrow heads, an odd window
        _decode("window_draft", 8, 4, 6000, 500, 32, 8, 64, 4, 16, "f16", 777, 3),
        # one decode step of one request: its token's log probability and the five best
        _score("score_one", 1, 32000, "bf16", 5),
        # a prompt's tokens scored, its padding left out
        _score("score_prompt", 2048, 32000, "bf16", 0, ignored=0.1),
        # fp32 logits of an odd vocabulary, some of it banned, read out of wider rows, twenty alternatives
        _score("score_odd", 333, 50021, "f32", 20, pad=3, banned=0.05),
        # a loss over log probabilities and entropy with its gradient, a large vocabulary
        _score("score_grad", 1024, 131072, "bf16", 0, grad=True, ignored=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "decode", "score"])
    bits, page, D = rng.choice([4, 8]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    window, sinks = _log(rng, 16, 8192), rng.choice([0, 1, 4, 16, 64])
    if op == "chunk":
        hq, hkv = rng.choice([(32, 32), (40, 40), (64, 8), (16, 4), (24, 2), (12, 4)])
        B, new = _log(rng, 1, 12), _log(rng, 1, 2048)
        past = _log(rng, 1, 30720) - 1
        while B * (past + new) * hkv * D > 130_000_000:
            B, past = (B + 1) // 2, past // 2
        if rng.random() < 0.6:
            window = sinks = 0
        c = _chunk("", B, new, past, hq, hkv, D, bits, page, dtype, window, sinks)
    elif op == "decode":
        hkv = rng.choice([2, 4, 8, 8, 32, 40])
        hq = hkv * rng.choice([1, 4, 8] if hkv <= 8 else [1])
        B, T = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 5])
        longest = _log(rng, 16, max(17, min(131072, 130_000_000 // (B * hkv * D))))
        c = _decode("", B, T, longest, rng.choice([T, max(T, longest // 2), longest]), hq, hkv, D, bits, page, dtype, window, sinks)
    else:
        V = rng.choice([32000, 65536, 131072, _log(rng, 300, 131072)])
        n = _log(rng, 1, min(4096, 130_000_000 // V))
        c = _score("", n, V, rng.choice(["bf16", "f16", "f32"]), rng.choice([0, 0, 1, 5, 20]), rng.random() < 0.4,
                   rng.choice([0, 0, 8, 3]), rng.choice([0.0, 0.1]), rng.choice([0.0, 0.05]))
    del c["name"]
    return c


# ---- what a user has in hand --------------------------------------------------------

def _tile_bytes(D, bits):
    return TILE * (2 * D * bits // 8 + 2 * (D // GROUP) * 4)


def _spread(n, most, least):
    """n whole numbers from most down to least, evenly."""
    return [most - (most - least) * i // max(1, n - 1) for i in range(n)]


def _requests(case):
    """(new, past) of each request, before the seed orders them."""
    B = case["B"]
    if case["op"] == "decode":
        return [(case["T"], max(0, n - case["T"])) for n in _spread(B, case["longest"], max(case["T"], case["shortest"]))]
    past = _spread(B, case["past"], 0)
    turned = [past[(i * 5) % B] if math.gcd(5, B) == 1 else past[i] for i in range(B)]
    return list(zip(_spread(B, case["new"], 1), turned))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "score":
        n, V = case["n"], case["V"]
        # logits of a model that is sure of some tokens and not of others
        x = randn(n, V + case["pad"]) * (1.0 + 2.0 * torch.rand((n, 1), generator=g, device="cuda"))
        tokens = torch.randint(0, V, (n,), generator=g, device="cuda")
        x[torch.arange(n, device="cuda"), tokens] += 8.0 * torch.rand(n, generator=g, device="cuda")
        if case["banned"]:
            ban = torch.rand((1, V + case["pad"]), generator=g, device="cuda") < case["banned"]
            ban = ban.expand(n, -1).clone()
            ban[torch.arange(n, device="cuda"), tokens] = False
            x.masked_fill_(ban, -math.inf)
        if case["ignored"]:
            tokens = torch.where(torch.rand(n, generator=g, device="cuda") < case["ignored"], -1, tokens)
        st["logits"], st["tokens"] = x.to(DT[case["dtype"]])[:, :V], tokens
        if case["grad"]:
            st["d_logprob"], st["d_entropy"] = -torch.rand(n, generator=g, device="cuda"), 0.1 * randn(n)
        return st
    D, bits, page, hkv, B = case["D"], case["bits"], case["page"], case["hkv"], case["B"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(int(seed))).tolist()
    each = _requests(case)
    new, lens = [each[i][0] for i in order], [sum(each[i]) for i in order]
    per = -(-max(lens) // page)
    pages, tb = B * per, _tile_bytes(D, bits)
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
    st["block_table"] = torch.randperm(pages, generator=g, device="cuda").int().view(B, per)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["host_lens"], st["host_new"] = lens, new
    if case["op"] == "decode":
        st["q"] = randn(B, case["T"], case["hq"], D).to(DT[case["dtype"]])
    else:
        at = [0]
        for n in new:
            at.append(at[-1] + n)
        st["starts"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        st["q"] = randn(at[-1], case["hq"], D).to(DT[case["dtype"]])
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
    _, h = _handle()
    c = st["case"]
    if c["op"] == "decode":
        return h.kv_attention(st["q"], _cache(st), st["block_table"], st["lens"], window=c["window"], sinks=c["sinks"])
    if c["op"] == "chunk":
        return h.kv_attention_chunk(st["q"], _cache(st), st["block_table"], st["lens"], st["starts"],
                                    window=c["window"] or None, sinks=c["sinks"])
    if c["grad"]:
        x = st["logits"].detach().requires_grad_()
        logprob, entropy, ids, alternatives = h.token_logprobs(x, st["tokens"], top=c["top"])
        d, = torch.autograd.grad([logprob, entropy], [x], [st["d_logprob"], st["d_entropy"]])
        out = [logprob.detach(), entropy.detach(), d]
    else:
        logprob, entropy, ids, alternatives = h.token_logprobs(st["logits"], st["tokens"], top=c["top"])
        out = [logprob, entropy]
    return out + [ids, alternatives.detach()] if c["top"] else out


def run(st):
    if own:
        return _run_own(st)
    return {"decode": _plain_decode, "chunk": _plain_chunk, "score": _plain_score}[st["case"]["op"]](st)


# ---- the plain forms ----------------------------------------------------------------

def _unpacked(t, D, bits):
    """Tiles [..., bytes] -> keys and values [..., 16, D] in 32 bits."""
    G, kb, per = D // GROUP, TILE * D * bits // 8, 32 // bits
    lead = t.shape[:-1]
    shift = torch.arange(0, 32, bits, device=t.device, dtype=torch.int32)

    def codes(o):      # [..., row (8), column (4), word of the lane, code of the word]
        w = t[..., o:o + kb].contiguous().view(torch.int32).view(*lead, -1, 32, 4).transpose(-3, -2).reshape(*lead, 8, 4, -1)
        return (w[..., None] >> shift) & (2 ** bits - 1)

    def meta(i, *shape):
        o = 2 * kb + 2 * TILE * G * i
        return t[..., o:o + 2 * TILE * G].contiguous().view(torch.float16).view(*lead, *shape).float()

    d = len(lead)
    at = lambda *order: tuple(range(d)) + tuple(d + o for o in order)  # noqa: E731
    k = codes(0).view(*lead, 8, 4, 2, G, 8 // per, per).permute(at(2, 0, 3, 1, 4, 5)).reshape(*lead, TILE, G, GROUP)
    k = k * meta(0, TILE, G)[..., None] + meta(1, TILE, G)[..., None]
    W = D // 8 // per
    v = codes(kb).view(*lead, 8, 4, 2, 2, W, per).permute(at(2, 1, 3, 5, 4, 0)).reshape(*lead, TILE, G, GROUP)
    s, z = (meta(i, G, 4, 2, 2).permute(at(2, 1, 3, 0)).reshape(*lead, TILE, G, 1) for i in (2, 3))
    return k.flatten(-2), (v * s + z).flatten(-2)


def _visible(at, pos, c):
    """Which tokens `at` a query at position `pos` sees (they broadcast)."""
    seen = at <= pos
    if c["window"]:
        seen = seen & ((at > pos - c["window"]) | (at < c["sinks"]))
    return seen


def _softmax(score, v, product):
    """Softmax over the last dimension, its product with the values, and the log-sum-exp."""
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    return torch.einsum(product, p, v) / total, (top + torch.log(total))[..., 0]


def _plain_decode(st):
    c = st["case"]
    B, T, hq, hkv, D, page = c["B"], c["T"], c["hq"], c["hkv"], c["D"], c["page"]
    q = st["q"].float().view(B, T, hkv, hq // hkv, D) * D ** -0.5
    # the tiles that hold anything seen: those of the sinks, then those from the first row's window on
    length = st["lens"][:, None].long()
    sunk = -(-c["sinks"] // TILE)
    first = ((length - T + 1 - c["window"]).clamp(min=0) // TILE).clamp(min=sunk)
    n = min(-(-(c["window"] + T) // TILE) + 1, -(-max(st["host_lens"]) // TILE))
    tiles = torch.cat([torch.arange(sunk, device=q.device).expand(B, -1), first + torch.arange(n, device=q.device)], 1)
    last = st["block_table"].shape[1] * page // TILE - 1
    used = tiles.clamp(max=last)
    pages = torch.gather(st["block_table"], 1, used // (page // TILE)).long()
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in _unpacked(st["pages"][pages, :, used % (page // TILE)], D, c["bits"]))
    at = (tiles[:, :, None] * TILE + torch.arange(TILE, device=q.device)).flatten(1)[:, None]
    pos = length[:, :, None] - T + torch.arange(T, device=q.device)[:, None]
    mask = _visible(at, pos, c)[:, :, None, None]
    score = torch.einsum("bthgd,bhnd->bthgn", q, k).masked_fill(~mask, -math.inf)
    o, lse = _softmax(score, v, "bthgn,bhnd->bthgd")
    return [o.reshape(B, T, hq, D).to(st["q"].dtype), lse.reshape(B, T, hq)]


def _plain_chunk(st):
    c = st["case"]
    hq, hkv, D, page = c["hq"], c["hkv"], c["D"], c["page"]
    out, lse, row = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], device="cuda"), 0
    for b, (T, n) in enumerate(zip(st["host_new"], st["host_lens"])):
        pages = st["block_table"][b, :-(-n // page)].long()
        pos = n - T + torch.arange(T, device="cuda")[:, None, None]
        seen = _visible(torch.arange(n, device="cuda"), pos, c)
        for h in range(hkv):
            k, v = (x.flatten(0, 2)[:n] for x in _unpacked(st["pages"][pages, h], D, c["bits"]))
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            q = st["q"][row:row + T, mine].float() * D ** -0.5
            score = torch.einsum("tgd,nd->tgn", q, k).masked_fill_(~seen, -math.inf)
            o, l = _softmax(score, v, "tgn,nd->tgd")
            out[row:row + T, mine], lse[row:row + T, mine] = o.to(out.dtype), l
        row += T
    return [out, lse]


def _plain_score(st):
    c = st["case"]
    x, kept = st["logits"].float(), st["tokens"] >= 0
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    log_total = torch.log(total)
    far = torch.where(e > 0, x - top, torch.zeros_like(x))
    entropy = (log_total - (e * far).sum(-1, keepdim=True, dtype=torch.float64) / total)
    at = st["tokens"].clamp(min=0)[:, None]
    logprob = torch.gather(x, 1, at).double() - top - log_total
    out = [torch.where(kept, logprob[:, 0], 0.0).float(), entropy[:, 0].float()]
    if c["grad"]:
        p = e / total.float()
        dl, de = torch.where(kept, st["d_logprob"], 0.0)[:, None], st["d_entropy"][:, None]
        d = -p * (dl + de * (far - log_total.float() + entropy.float()))
        d.scatter_add_(1, at, dl)
        out.append(d.to(st["logits"].dtype))
    if c["top"]:
        best, ids = (t[:, :c["top"]] for t in torch.sort(x, descending=True, stable=True))
        out += [ids, (best - top - log_total).float()]
    return out


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    c = case
    e = DT[c["dtype"]].itemsize
    if c["op"] == "score":
        # (a gradient needs the row's sums first: the logits are read twice, as no on-chip memory holds them all)
        b = c["n"] * c["V"] * e * (3.0 if c["grad"] else 1.0) + c["n"] * (16.0 + 12 * c["top"])
        return {"bytes": b, "flops": c["n"] * c["V"] * (12.0 if c["grad"] else 6.0)}
    kept = pairs = rows = 0
    for T, past in _requests(c):
        rows += T
        # tokens that the rows at `past` and after see, summed, and those that any of them sees
        W, S = c["window"] or past + T, c["sinks"]
        for p in range(past, past + T):
            pairs += min(p + 1, W) + min(S, max(0, p + 1 - W))
        before = max(0, past + 1 - W)
        kept += past + T - before + min(S, before)
    held = c["hkv"] * _tile_bytes(c["D"], c["bits"]) / TILE          # bytes a token holds in the cache
    b = held * kept + rows * c["hq"] * (2.0 * c["D"] * e + 4)
    return {"bytes": float(b), "flops": 4.0 * c["D"] * c["hq"] * pairs}


# ---- the definitions in 64 bits -----------------------------------------------------

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


def _exact_score(st):
    c = st["case"]
    x, tokens = st["logits"].double(), st["tokens"]
    log_p = torch.log_softmax(x, -1)
    p = log_p.exp()
    entropy = -torch.xlogy(p, p).sum(-1)
    given = torch.where(tokens >= 0, log_p[torch.arange(c["n"], device="cuda"), tokens.clamp(min=0)], 0.0)
    out = [given, entropy]
    if c["grad"]:
        de = st["d_entropy"].double()[:, None]
        d = -de * (torch.xlogy(p, p) + p * entropy[:, None])
        for i in range(c["n"]):
            if int(tokens[i]) >= 0:
                w = float(st["d_logprob"][i])
                d[i] -= w * p[i]
                d[i, tokens[i]] += w
        out.append(d)
    if c["top"]:
        # one number per logit in the order wanted: the value's bits as a whole number, then the lower index
        b = st["logits"].float().contiguous().view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7fffffff), b)
        key = b * (1 << 20) - torch.arange(c["V"], device="cuda")
        ids = torch.topk(key, c["top"], dim=-1).indices
        out += [ids, torch.gather(log_p, 1, ids)]
    return out


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "score":
        return _exact_score(st)
    hq, hkv, D, page = c["hq"], c["hkv"], c["D"], c["page"]
    rows = sum(st["host_new"])
    q = st["q"].reshape(rows, hq, D).double()
    out = torch.zeros((rows, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, hq), dtype=torch.float64, device="cuda")
    for h in range(hkv):
        row = 0
        for b, (T, n) in enumerate(zip(st["host_new"], st["host_lens"])):
            # a window's tokens lie in the sinks and in the last tokens: two runs of pages
            low = max(0, n - T + 1 - c["window"]) // page if c["window"] else 0
            sunk = min(low, -(-c["sinks"] // page))
            used = list(range(sunk)) + list(range(low, -(-n // page)))
            at = torch.cat([torch.arange(page, device="cuda") + i * page for i in used])
            k, v = _values64(st["pages"][st["block_table"][b, used].long(), h].flatten(0, 1), D, c["bits"])
            v = torch.where(at[:, None] < n, v, 0.0)
            heads = range(h * (hq // hkv), (h + 1) * (hq // hkv))
            for t0 in range(0, T, 256):
                t1 = min(T, t0 + 256)
                pos = n - T + torch.arange(t0, t1, device="cuda")[:, None]
                hidden = at[None] > pos
                if c["window"]:
                    hidden |= (at[None] <= pos - c["window"]) & (at[None] >= c["sinks"])
                for i in heads:
                    s = ((q[row + t0:row + t1, i] @ k.T) * D ** -0.5).masked_fill(hidden, -math.inf)
                    lse[row + t0:row + t1, i] = torch.logsumexp(s, -1)
                    out[row + t0:row + t1, i] = torch.softmax(s, -1) @ v
            row += T
    return [out.view(st["q"].shape), lse.view(st["q"].shape[:-1])]
