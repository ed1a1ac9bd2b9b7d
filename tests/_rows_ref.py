"""Attention of any number of new rows per request over the low-bit cache, with windows and sinks, restated plainly in 64
bits over the cache's own values.  Shared by the tests of sliding windows and of token chunks.

Bounds, with u = 2^-11 the relative rounding of a binary16:
* a score is off by at most 2^-20 * scale * sum_d |q_d k_jd| (fp32 sums of D products, and the exponential's 2^-22), so lse by
  the largest such amount plus 2^-19, and each probability by twice that, relatively;
* a probability is rounded by u.  lq_kv_attention: P S against c and P against Z, each by u, with |S c| <= |v| + |Z|, so
  u (|v| + 2 |Z|) per unit of probability (its half-step figure u / 2 twice).  lq_kv_attention_chunk: the value itself by u,
  or by 2^-25 below 2^-14, and P by u, for binary16 outputs (which multiply what that left out too) by u^2;
* lq_kv_attention holds P in units of 2^-11, lq_kv_attention_chunk of 2^-8; below 2^-14 it is a subnormal binary16, off by
  2^-25: 2^-36 and 2^-33 of a value's size for each of n keys;
* the output's own rounding: 2^-8 of it for bfloat16, 2^-11 for binary16.
"""
from __future__ import annotations

import numpy as np

from tests import _kv_ref as R


def visible(n, fresh, window, sinks):
    """[fresh][n]: whether new row t of a request of n tokens sees token j."""
    p = n - fresh + np.arange(fresh)[:, None]
    j = np.arange(n)[None]
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attend(q, k, v, seen, scale):
    """q [T][g][D], k and v [n][D], seen [T][n].  out [T][g][D], lse [T][g], sum_j p_j |v_j|, max_j sum_d |q_d k_jd|."""
    T, g, D = q.shape
    out, mass = np.zeros((T, g, D)), np.zeros((T, g, D))
    lse, size = np.full((T, g), -np.inf), np.zeros((T, g))
    some = seen.any(1)
    if not some.any():
        return out, lse, mass, size
    any_ = seen.any(0)                                   # (what no row sees may be anything)
    k, v, seen = k[any_].astype(np.float64), v[any_].astype(np.float64), seen[:, any_]
    with np.errstate(invalid="ignore"):
        s = np.einsum("tgd,nd->tgn", q.astype(np.float64), k) * scale
    s = np.where(seen[:, None], s, -np.inf)
    top = np.where(some[:, None, None], s.max(-1, keepdims=True), 0.0)
    p = np.exp(s - top)
    l = np.where(some[:, None, None], p.sum(-1, keepdims=True), 1.0)
    p = p / l
    lse = np.where(some[:, None], (top + np.log(l))[..., 0], -np.inf)
    out, mass = p @ v, p @ np.abs(v)
    for i in range(g):
        size[:, i] = np.where(seen, np.abs(q[:, i].astype(np.float64)) @ np.abs(k).T, 0.0).max(-1)
    return out, lse, mass, size


class Rows:
    """A cache of random pages with every token that no row sees NaN or infinite, shuffled page lists, and packed new rows."""

    def __init__(self, lqm, fresh, lens, hq=8, hkv=2, D=128, bits=4, page=64, dtype="bf16", window=0, sinks=0, seed=0, extra_pages=0,
                 spread=1.0, lead=0, tail=0, pages=None, poison=True):
        import torch
        g = np.random.default_rng(seed)
        self.fresh, self.lens, self.hq, self.hkv, self.D, self.bits, self.page = fresh, lens, hq, hkv, D, bits, page
        self.window, self.sinks, self.scale = window, sinks, D ** -0.5
        B, G, top = len(lens), D // 32, 2 ** bits - 1
        each = pages or max(1, -(-max(lens) // page)) + extra_pages
        self.capacity = each * page
        total = B * each + 1
        shape = (total, hkv, page // 16, 16)
        codes = [g.integers(0, top + 1, shape + (D,), dtype=np.uint8) for _ in range(2)]
        meta = []
        for scale in (spread, 1.0):
            S = ((g.random(shape + (G,)) + 3.0) * scale / top).astype(np.float16)
            Z = (-0.5 * top * S.astype(np.float32) + 0.3 * scale * g.standard_normal(shape + (G,))).astype(np.float16)
            meta += [S, Z]
        self.bt = g.permutation(total).astype(np.int32)[:B * each].reshape(B, each)
        if poison:
            used = np.zeros((total, page), bool)
            for b in range(B):
                n = self.length(b)
                j = np.nonzero(visible(n, fresh[b], window, sinks).any(0))[0]
                used[self.bt[b][j // page], j % page] = True
            free = ~used.reshape(total, 1, page // 16, 16)
            for i, m in enumerate(meta):
                m[np.broadcast_to(free, shape)] = [np.nan, np.inf, np.nan, -np.inf][i]
        self.codes, self.meta = codes, meta
        self.starts = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32) + lead
        n = int(self.starts[-1]) + tail
        dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.q = torch.from_numpy(g.standard_normal((n, hq, D)).astype(np.float32)).to(dt).cuda()
        self.dev = dict(bt=torch.from_numpy(self.bt).cuda(), starts=torch.from_numpy(self.starts).cuda(),
                        lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        tiles = R.pack(codes[0], meta[0], meta[1], codes[1], meta[2], meta[3], bits)
        self.cache = lqm.KVCache(torch.from_numpy(tiles).cuda(), page_size=page, kv_heads=hkv, head_dim=D, bits=bits)
        self.values()

    def values(self):
        m, (total, hkv) = self.meta, self.codes[0].shape[:2]
        with np.errstate(all="ignore"):
            self.k = R.dequantize(self.codes[0], m[0], m[1]).reshape(total, hkv, self.page, self.D)
            self.v = R.dequantize(self.codes[1], m[2], m[3]).reshape(total, hkv, self.page, self.D)
        self.z = np.repeat(np.abs(m[3].astype(np.float32)), 32, -1).reshape(total, hkv, self.page, self.D)

    def repack(self):
        import torch
        m = self.meta
        self.cache.pages.copy_(torch.from_numpy(R.pack(self.codes[0], m[0], m[1], self.codes[1], m[2], m[3], self.bits)))
        self.values()

    def where(self, b, j):
        """Indices of token j of request b in the codes and scales: page, tile, place in the tile (heads lie between)."""
        return self.bt[b][j // self.page], j % self.page // 16, j % 16

    def length(self, b):
        return min(max(self.lens[b], 0), self.capacity)

    def chunk(self, handle, **kw):
        d = self.dev
        return handle.kv_attention_chunk(kw.pop("q", self.q), self.cache, d["bt"], d["lens"], d["starts"], scale=self.scale,
                                         window=self.window or None, sinks=self.sinks, **kw)

    def decode(self, handle, **kw):
        """The same rows by kv_attention: every request has as many."""
        d, T = self.dev, self.fresh[0]
        q = self.q.view(len(self.lens), T, self.hq, self.D)
        o, lse = handle.kv_attention(q, self.cache, d["bt"], d["lens"], scale=self.scale, window=self.window or None,
                                     sinks=self.sinks, **kw)
        return o.reshape(self.q.shape), lse.reshape(self.q.shape[:2])

    def check(self, out, lse, dense=True, requests=None):
        import torch
        ulp = 2.0 ** -8 if self.q.dtype == torch.bfloat16 else 2.0 ** -11
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        q, gs = self.q.float().cpu().numpy(), self.hq // self.hkv
        worst = 0.0
        for b in (range(len(self.lens)) if requests is None else requests):
            n, rows = self.length(b), slice(self.starts[b], self.starts[b + 1])
            if self.fresh[b] == 0:
                continue
            j = np.arange(n)
            pages, offs = self.bt[b][j // self.page], j % self.page
            seen = visible(n, self.fresh[b], self.window, self.sinks)
            for h in range(self.hkv):
                hs = slice(h * gs, (h + 1) * gs)
                k, v, z = self.k[pages, h, offs], self.v[pages, h, offs], self.z[pages, h, offs]
                o, s, mass, size = attend(q[rows, hs], k, v, seen, self.scale)
                size = size * self.scale
                got, got_lse = out[rows, hs], lse[rows, hs]
                assert np.array_equal(np.isneginf(got_lse), np.isneginf(s)), (b, h)
                live = ~np.isneginf(s)
                e = np.abs(got_lse[live] - s[live])
                assert np.all(e <= 2.0 ** -20 * size[live] + 2.0 ** -19), (b, h, e.max())
                most = np.abs(v[seen.any(0)]).max() if seen.any() else 0.0
                if dense:
                    of_p = 2.0 ** -11 if ulp > 2.0 ** -11 else 2.0 ** -22
                    bound = (2.0 ** -11 + of_p + 2.0 ** -22 + 2.0 ** -18 * (1 + size[..., None])) * mass + 2.0 ** -25
                else:
                    zmass = attend(q[rows, hs], k, z, seen, self.scale)[0]
                    bound = (2.0 ** -11 + 2.0 ** -18 * (1 + size[..., None])) * (mass + 2 * zmass)
                bound = bound + ulp * np.abs(o) + (2.0 ** -24 + n * 2.0 ** (-33 if dense else -36)) * most
                err = np.abs(got - o)
                worst = max(worst, float((err / (bound + 1e-30)).max()))
                assert np.all(err <= bound + 1e-30), (b, h, float((err / (bound + 1e-30)).max()))
                assert np.all(got[~live] == 0)
        return worst
