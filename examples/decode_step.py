"""The attention block of a decoder layer, one decode step after another, all of it on low-bit storage.

    q, k, v = x Wq', x Wk', x Wv'        2-bit weights, one grouped launch
    q, k rotated, k and v into the cache  4-bit pages, one launch
    attention over the cache              the system prompt's pages shared by all requests
    y = o Wo'                             2-bit weights

The requests share a prefix (a system prompt), which was written once; each request's own tokens lie in
pages of its own.  Run it on a GPU:  python examples/decode_step.py
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import bit_weight_quantized_dequant_gb300 as lq
import synth


class AttentionBlock:
    """Low-bit projections, a rotation table, a cache and the page lists of a batch of requests."""

    def __init__(self, handle, hidden, q_heads, kv_heads, head_dim, batch, pages_each, prefix_pages, page_size=64, bits=4,
                 seed=0, max_positions=4096):
        self.h, self.q_heads, self.kv_heads, self.dim = handle, q_heads, kv_heads, head_dim

        def weights(n, k, i):
            anchors = 8 if k <= 1024 else 32
            return lq.QuantWeights.from_host(synth.random_packed_2bit(n, k, anchors, seed=seed, matrix_id=i), lq.FMT_2BIT)

        self.wq, self.wk = weights(q_heads * head_dim, hidden, 0), weights(kv_heads * head_dim, hidden, 1)
        self.wv, self.wo = weights(kv_heads * head_dim, hidden, 2), weights(hidden, q_heads * head_dim, 3)
        self.table = handle.rope_table(max_positions, head_dim, factor=4.0, original_length=1024.0)
        pages = batch * pages_each + prefix_pages
        self.cache = lq.KVCache(num_pages=pages, page_size=page_size, kv_heads=kv_heads, head_dim=head_dim, bits=bits)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int().cuda()
        self.block_table = order[:batch * pages_each].view(batch, pages_each)
        self.prefix_table, self.prefix_len = order[batch * pages_each:], 0
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def slots(self, tokens):
        """Slots of each request's own tokens number `tokens` [batch]."""
        ps = self.cache.page_size
        page = torch.gather(self.block_table, 1, (tokens // ps).long()[:, None])[:, 0]
        return page.long() * ps + tokens % ps

    def write_prefix(self, k, v):
        """A prefill's keys and values of the shared prompt, already projected: [n][kv_heads][dim]."""
        n, ps = k.shape[0], self.cache.page_size
        at = torch.arange(n, device="cuda")
        slots = self.prefix_table[at // ps].long() * ps + at % ps
        self.h.kv_append(self.cache, k, v, slots, table=self.table, positions=at.int())
        self.prefix_len = n

    def step(self, x):
        """x [batch][hidden], the next token of every request: the block's output, one token longer a cache."""
        batch, h = x.shape[0], self.h
        q, k, v = (torch.empty((batch, w.N), dtype=x.dtype, device=x.device) for w in (self.wq, self.wk, self.wv))
        h.gemv_grouped([h.problem(w, x, y) for w, y in ((self.wq, q), (self.wk, k), (self.wv, v))])
        heads = lambda t, n: t.view(batch, n, self.dim)  # noqa: E731
        slots, positions = self.slots(self.lens), self.lens + self.prefix_len
        q = h.kv_append(self.cache, heads(k, self.kv_heads), heads(v, self.kv_heads), slots, q=heads(q, self.q_heads),
                        table=self.table, positions=positions)
        self.lens += 1
        o, _ = h.kv_attention(q[:, None], self.cache, self.block_table, self.lens, prefix_table=self.prefix_table,
                              prefix_len=self.prefix_len)
        return h.gemv(self.wo, o.view(batch, -1), y_dtype=x.dtype)


def main(batch=4, steps=8, prefix=300):
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    with lq.Handle(0) as h:
        block = AttentionBlock(h, hidden=1024, q_heads=16, kv_heads=4, head_dim=128, batch=batch, pages_each=2, prefix_pages=5)
        block.write_prefix(randn(prefix, 4, 128), randn(prefix, 4, 128))
        for _ in range(steps):
            y = block.step(randn(batch, 1024))
        h.sync()
        print(f"{batch} requests, {prefix} shared tokens, {int(block.lens[0])} of their own: output {tuple(y.shape)}, "
              f"|y| = {float(y.float().norm()):.3f}; the cache holds {block.cache.pages.numel() / 1e6:.2f} MB")
    return y


if __name__ == "__main__":
    main()
