"""A prompt scored and continued through one attention block, all of it on low-bit storage.

    q, k, v = x Wq', x Wk', x Wv'          2-bit weights, each chunk's rows at once
    q, k rotated, k and v into the cache   4-bit pages
    attention of the chunk over the cache  all of it, or a window with sinks
    logits = (x + o Wo') H'                a low-bit head
    log probabilities of the next tokens   with the entropy of each position

The prompt goes through in chunks of any size.  Afterwards single tokens follow: each is the best alternative of the
step before.  Run it on a GPU:  python examples/score_prompt.py
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


class Scorer:
    """Random low-bit weights of one attention block and a head, and a cache for one request."""

    def __init__(self, handle, vocab=2048, hidden=512, q_heads=8, kv_heads=2, head_dim=128, pages=40, page_size=64, window=None,
                 sinks=0, seed=0):
        self.h, self.q_heads, self.kv_heads, self.dim = handle, q_heads, kv_heads, head_dim
        self.window, self.sinks, self.length = window, sinks, 0

        def weights(n, k, i):
            return lq.QuantWeights.from_host(synth.random_packed_2bit(n, k, 8, seed=seed, matrix_id=i), lq.FMT_2BIT)
        self.wq, self.wk = weights(q_heads * head_dim, hidden, 0), weights(kv_heads * head_dim, hidden, 1)
        self.wv, self.wo = weights(kv_heads * head_dim, hidden, 2), weights(hidden, q_heads * head_dim, 3)
        self.head = weights(vocab, hidden, 4)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda").bfloat16()
        self.table = handle.rope_table(pages * page_size, head_dim)
        self.cache = lq.KVCache(num_pages=pages, page_size=page_size, kv_heads=kv_heads, head_dim=head_dim, bits=4)
        self.block_table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int().cuda()[None]

    def project(self, w, x):
        """x w': a decode product for few rows, a prefill product for many."""
        return self.h.gemv(w, x, y_dtype=x.dtype) if len(x) <= 32 else self.h.gemm(w, x, y_dtype=x.dtype)

    def logits(self, tokens):
        """Logits after each of the next `tokens` (int64 [n]) of the request; fp32 [n][vocab]."""
        h, n = self.h, len(tokens)
        x = self.embedding[tokens]
        heads = lambda w, k: self.project(w, x).view(n, k, self.dim)  # noqa: E731
        at = torch.arange(self.length, self.length + n, device="cuda")
        slots = self.block_table[0][at // self.cache.page_size].long() * self.cache.page_size + at % self.cache.page_size
        q = h.kv_append(self.cache, heads(self.wk, self.kv_heads), heads(self.wv, self.kv_heads), slots, q=heads(self.wq, self.q_heads),
                        table=self.table, positions=at.int())
        self.length += n
        lens = torch.full((1,), self.length, dtype=torch.int32, device="cuda")
        if n == 1:
            o, _ = h.kv_attention(q[:, None], self.cache, self.block_table, lens, window=self.window, sinks=self.sinks)
        else:
            starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            o, _ = h.kv_attention_chunk(q, self.cache, self.block_table, lens, starts, window=self.window, sinks=self.sinks)
        y = x + self.project(self.wo, o.reshape(n, -1))
        w = self.head
        return h.gemv(w, y, y_dtype=torch.float32) if n <= 32 else h.gemm(w, y, y_dtype=torch.float32)

    def score(self, tokens, chunk):
        """Log probability of each token of a prompt given those before it (of the first: none), and the last logits."""
        out = []
        for i in range(0, len(tokens), chunk):
            part = tokens[i:i + chunk]
            follows = torch.cat([tokens[i + 1:i + chunk + 1], tokens.new_full((max(0, i + chunk + 1 - len(tokens)),), -1)])[:len(part)]
            logits = self.logits(part)
            out.append(self.h.token_logprobs(logits, follows)[:2])
        return torch.cat([p for p, _ in out])[:-1], torch.cat([e for _, e in out]), logits[-1:]

    def continue_with(self, logits, steps):
        """The best token of each step, taken, with its log probability."""
        tokens, scores = [], []
        for _ in range(steps):
            _, _, ids, best = self.h.token_logprobs(logits, torch.full((1,), -1, dtype=torch.int64, device="cuda"), top=5)
            tokens.append(ids[:, 0])
            scores.append(best[:, 0])
            logits = self.logits(ids[:, 0])
        return torch.cat(tokens), torch.cat(scores)


def main(length=700, chunk=256, steps=4, window=128, sinks=4):
    with lq.Handle(0) as h:
        s = Scorer(h, window=window, sinks=sinks)
        prompt = torch.randint(0, len(s.embedding), (length,), generator=torch.Generator().manual_seed(1)).cuda()
        logprob, entropy, logits = s.score(prompt, chunk)
        tokens, scores = s.continue_with(logits, steps)
        h.sync()
        print(f"{length} tokens in chunks of {chunk}: mean log probability {float(logprob.mean()):.3f}, mean entropy "
              f"{float(entropy.mean()):.3f}; then {tokens.tolist()} at {[round(float(x), 3) for x in scores]}")
    return logprob, tokens


if __name__ == "__main__":
    main()
