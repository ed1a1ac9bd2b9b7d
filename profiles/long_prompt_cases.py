"""The calls behind long_prompt.md, three of each:  python profiles/long_prompt_cases.py CASE"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch

import bit_weight_quantized_dequant_gb300 as lq


def cache(h, requests, tokens, kv_heads, bits, page):
    each = -(-tokens // page)
    c = lq.KVCache(num_pages=requests * each, page_size=page, kv_heads=kv_heads, head_dim=128, bits=bits)
    n = c.num_pages * page
    for first in range(0, n, 65536):
        at = torch.arange(first, min(n, first + 65536), device="cuda")
        k, v = (torch.randn(len(at), kv_heads, 128, device="cuda").bfloat16() for _ in range(2))
        h.kv_append(c, k, v, at)
    return c, torch.randperm(c.num_pages, device="cuda").int().view(requests, each)


def main(case):
    h = lq.Handle(0)
    torch.manual_seed(0)
    if case == "chunk":         # 512 tokens at the end of 8 Ki, 64 query heads over 8, 4 bits
        c, table = cache(h, 1, 8192, 8, 4, 64)
        q = torch.randn(512, 64, 128, device="cuda").bfloat16()
        lens, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([8192], [0, 512]))
        for _ in range(3):
            h.kv_attention_chunk(q, c, table, lens, starts)
    elif case == "window":      # 32 requests of 100 .. 5001 tokens, 40 heads, 8 bits, a window of 1024 and 16 sinks
        c, table = cache(h, 32, 5001, 40, 8, 32)
        q = torch.randn(32, 1, 40, 128, device="cuda").bfloat16()
        lens = torch.tensor([5001 - 4901 * i // 31 for i in range(32)], dtype=torch.int32, device="cuda")
        for _ in range(3):
            h.kv_attention(q, c, table, lens, window=1024, sinks=16)
    elif case in ("score", "top", "grad"):   # 2048 rows of 32000 bf16 logits; 333 of 50021 fp32 with 20 alternatives; the gradient
        n, V, dtype, top = (333, 50021, torch.float32, 20) if case == "top" else (2048, 32000, torch.bfloat16, 0)
        x = torch.randn(n, V, device="cuda").mul_(2.0).to(dtype).requires_grad_(case == "grad")
        t = torch.randint(0, V, (n,), device="cuda")
        for _ in range(3):
            logprob, entropy, _, _ = h.token_logprobs(x, t, top=top)
            if case == "grad":
                torch.autograd.grad([logprob, entropy], [x], [torch.ones_like(logprob), torch.ones_like(entropy)])
    h.sync()


if __name__ == "__main__":
    main(sys.argv[1])
