"""A plain restatement, in numpy, of the rotary, cache and attention definitions of include/lq.h.

Shared by the tests of those operators; nothing here touches the library.
"""
from __future__ import annotations

import numpy as np

GROUP, TILE = 32, 16


def frequencies(rot, base=10000.0, factor=1.0, original=0.0, low=1.0, high=32.0):
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    keep = np.zeros_like(f) if original == 0 else np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def table64(first, count, rot, mscale=1.0, **kw):
    a = np.arange(first, first + count, dtype=np.float64)[:, None] * frequencies(rot, **kw)
    return np.concatenate([np.cos(a), np.sin(a)], 1) * mscale


def rotate(x, table, positions, layout, inverse=False, dtype=np.float32):
    """x [n][H][D] in `dtype` arithmetic (fp32 gives the definition's own roundings)."""
    y = np.array(x, dtype=dtype)
    rot = table.shape[1]
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == 0 else (2 * i, 2 * i + 1)
    c = table[positions][:, None, :rot // 2].astype(dtype)
    s = table[positions][:, None, rot // 2:].astype(dtype)
    if inverse:
        s = -s
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - w * s, u * s + w * c
    return y


def quantize(x, bits):
    """x fp32 [..., D] -> codes uint8 [..., D], S and Z float16 [..., D / 32]; fp32 steps."""
    top = np.float32(2 ** bits - 1)
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        g = np.where(np.isnan(g), g, np.clip(g, np.float32(-65504), np.float32(65504)))
        lo, hi = g.min(-1), g.max(-1)                       # (numpy's min and max carry NaN)
        Z = lo.astype(np.float16)
        S = ((hi - lo) * (np.float32(1) / top)).astype(np.float16)
        s, z = S.astype(np.float32)[..., None], Z.astype(np.float32)[..., None]
        c = np.where(s > 0, np.clip(np.rint((g - z) / np.where(s > 0, s, np.float32(1))), 0, top), np.float32(0))
    return c.astype(np.uint8).reshape(x.shape), S, Z


def dequantize(c, S, Z):
    g = c.reshape(*c.shape[:-1], -1, GROUP).astype(np.float32)
    with np.errstate(invalid="ignore"):
        return (g * S.astype(np.float32)[..., None] + Z.astype(np.float32)[..., None]).reshape(c.shape)


def places(bits, D):
    """Bit offsets inside a tile of key and value codes [16][D], byte offsets of keys' and values' S [16][G]
    (their Z lie 16 * G * 2 bytes further)."""
    per, G = 32 // bits, D // GROUP
    wk, wv = D // (4 * per), D // (8 * per)
    t, d = np.arange(TILE)[:, None], np.arange(D)[None]
    region = TILE * D * bits // 8

    def bit(lane, q, e):
        return 8 * ((q // 4) * 512 + lane * 16 + (q % 4) * 4) + bits * e

    r = d % 32
    k = bit(4 * (t % 8) + r // 8, (t // 8) * wk + (d // 32) * (wk // G) + (r % 8) // per, r % per)
    slab = d // 8
    j = t % 2 + 2 * (t // 8)
    v = bit(4 * (d % 8) + (t % 8) // 2, j * wv + slab % wv, slab // wv) + 8 * region
    g = np.arange(G)[None]
    pos = 4 * ((t % 8) // 2) + t % 2 + 2 * (t // 8)
    ks = 2 * region + 2 * (t * G + g)
    vs = 2 * region + 2 * 2 * TILE * G + 2 * (g * TILE + pos)
    return k, v, ks, vs


def pack(kc, ks, kz, vc, vs, vz, bits):
    """Tiles [..., bytes] of codes [..., 16, D] and float16 S, Z [..., 16, G]."""
    D = kc.shape[-1]
    G = D // GROUP
    lead = kc.shape[:-2]
    out = np.zeros(lead + (TILE * (2 * D * bits // 8 + 8 * G),), np.uint8)
    pk, pv, ms, mv = places(bits, D)
    for c, p in ((kc, pk), (vc, pv)):
        for sub in range(8 // bits):                        # (a byte's nibbles one after the other)
            sel = (p % 8) == sub * bits
            out[..., p[sel] // 8] |= c[..., sel] << (sub * bits)
    for m, p in ((ks, ms), (kz, ms + 2 * TILE * G), (vs, mv), (vz, mv + 2 * TILE * G)):
        b = np.ascontiguousarray(m).view(np.uint8).reshape(*lead, TILE, G, 2)
        out[..., p], out[..., p + 1] = b[..., 0], b[..., 1]
    return out


def unpack(tiles, bits, D):
    """Tiles [..., bytes] -> keys and values fp32 [..., 16, D], with the codes, S and Z of both."""
    G = D // GROUP
    pk, pv, ms, mv = places(bits, D)

    def codes(p):
        return (tiles[..., p // 8] >> (p % 8).astype(np.uint8)) & np.uint8(2 ** bits - 1)

    def half(p):
        return np.stack([tiles[..., p], tiles[..., p + 1]], -1).view(np.float16)[..., 0]

    kc, vc = codes(pk), codes(pv)
    k = (kc, half(ms), half(ms + 2 * TILE * G))
    v = (vc, half(mv), half(mv + 2 * TILE * G))
    return dequantize(*k), dequantize(*v), k, v


def attend(q, keys, values, visible, scale):
    """One request and kv head in 64 bits: q [T][g][D], keys and values [n][D], visible [T] counts (the prefix
    included).  Returns out [T][g][D], lse [T][g], sum_j p_j |v_j| like out, and max_j sum_d |q_d k_jd| like lse."""
    T, g, D = q.shape
    out, lse = np.zeros((T, g, D)), np.full((T, g), -np.inf)
    mass, size = np.zeros((T, g, D)), np.zeros((T, g))
    for t in range(T):
        n = visible[t]
        if n <= 0:
            continue
        k, v, x = keys[:n].astype(np.float64), values[:n].astype(np.float64), q[t].astype(np.float64)
        s = x @ k.T * scale
        top = s.max(-1, keepdims=True)
        p = np.exp(s - top)
        l = p.sum(-1, keepdims=True)
        out[t], lse[t] = p @ v / l, (top + np.log(l))[:, 0]
        mass[t], size[t] = p @ np.abs(v) / l, (np.abs(x) @ np.abs(k).T).max(-1)
    return out, lse, mass, size
