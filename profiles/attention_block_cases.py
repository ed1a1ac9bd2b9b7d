"""The calls behind attention_block.md, three of each:  python profiles/attention_block_cases.py CASE"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch

import bit_weight_quantized_dequant_gb300 as lq


def attention(h, lens, q_heads, kv_heads, bits, page, prefix=0):
    batch, each, shared = len(lens), -(-max(lens) // page), -(-prefix // page)
    cache = lq.KVCache(num_pages=batch * each + shared, page_size=page, kv_heads=kv_heads, head_dim=128, bits=bits)
    n = cache.num_pages * page
    for first in range(0, n, 65536):
        at = torch.arange(first, min(n, first + 65536), device="cuda")
        k, v = (torch.randn(len(at), kv_heads, 128, device="cuda").bfloat16() for _ in range(2))
        h.kv_append(cache, k, v, at)
    order = torch.randperm(cache.num_pages, device="cuda").int()
    table, prefix_table = order[:batch * each].view(batch, each), order[batch * each:]
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(batch, 1, q_heads, 128, device="cuda").bfloat16()
    for _ in range(3):
        h.kv_attention(q, cache, table, lens, prefix_table=prefix_table if prefix else None, prefix_len=prefix)


def main(case):
    h = lq.Handle(0)
    torch.manual_seed(0)
    if case == "long":          # one request of 128 Ki tokens, 64 query heads over 8
        attention(h, [131072], 64, 8, 4, 64)
    elif case == "ragged":      # 24 requests, 1 .. 4001 tokens, 40 heads
        attention(h, [1 + 174 * i for i in range(23)] + [4001], 40, 40, 8, 32)
    elif case == "prefix":      # 48 requests of 1 .. 700 tokens over 32100 shared ones, 64 query heads over 8
        attention(h, [1 + 14 * i for i in range(47)] + [700], 64, 8, 4, 64, prefix=32100)
    elif case == "append":      # 2048 tokens of a prefill, rotation and cache write, 64 query heads, 8 kv heads
        cache = lq.KVCache(num_pages=2048 // 64, page_size=64, kv_heads=8, head_dim=128, bits=8)
        table = h.rope_table(131072, 128, factor=16.0, original_length=8192.0)
        k, v = (torch.randn(2048, 8, 128, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn(2048, 64, 128, device="cuda").bfloat16()
        at = torch.arange(2048, device="cuda")
        for _ in range(3):
            h.kv_append(cache, k, v, at, q=q, table=table, positions=at.int())
    h.sync()


if __name__ == "__main__":
    main(sys.argv[1])
