// Attention of a decode step (lq_attn_decode.cuh): the requests of a call, with the prefix they share.

#include "lq_attn_decode.cuh"

namespace lq {
namespace {

// Requests first .. first + n - 1 of a call, or with launch false whether the workspace has room for them at once.
// window 0: none.
lq_status attend(lq_handle h, const lq_kv_cache& c, const lq_kv_attention_args& a, int window, int sinks, int first, int n, bool launch,
                 cudaStream_t stream) {
    AttnParams P = {};
    P.window = window, P.sinks = sinks;
    P.cache = KvView{static_cast<uint8_t*>(c.pages), c.num_pages, c.page_size, c.kv_heads, c.page_size / kKvTile};
    const int64_t row0 = (int64_t)first * a.tokens;
    P.q = static_cast<const uint16_t*>(a.q) + row0 * a.q_token_stride, P.out = static_cast<uint16_t*>(a.out) + row0 * a.out_token_stride;
    P.lse = a.lse ? a.lse + row0 * a.q_heads : nullptr;
    P.q_stride = a.q_token_stride, P.out_stride = a.out_token_stride;
    P.tokens = a.tokens, P.q_heads = a.q_heads, P.group = a.q_heads / c.kv_heads;
    P.scale_log2 = a.scale * 1.4426950408889634f;
    P.counters = h->counters;
    P.status = h->status_flag;
    if ((int64_t)n * a.tokens * P.group > 0x7fffffffLL) return LQ_ERR_UNSUPPORTED;
    P.all_rows = n * a.tokens * P.group;
    P.page_shift = -1;
    for (int i = 0; i < 27; ++i)
        if (P.cache.tiles_per_page == 1 << i) P.page_shift = i;
    // workspace: what the prefix run leaves, then partial sums
    char* ws = reinterpret_cast<char*>(h->partials);
    const size_t cap = h->partial_floats * sizeof(float), rows = (size_t)c.kv_heads * P.all_rows;
    const bool bf16 = a.dtype == LQ_BF16;
    auto go = [&](AttnParams& p, size_t pre, bool now) {
        const Scratch s{ws + pre, cap - pre, 0, now, stream};
        if (pre > cap) return LQ_ERR_WORKSPACE;
        return p.window ? run_attn_window(h, p, c.bits, c.head_dim, bf16, s) : run_shape<false>(h, p, c.bits, c.head_dim, bf16, s);
    };
    AttnParams own = P;
    own.prefix = a.prefix_len > 0 ? 2 : 0;
    own.block_table = a.block_table + first * a.block_table_stride, own.bt_stride = a.block_table_stride, own.lens = a.lens + first;
    own.requests = n, own.rows = a.tokens * P.group, own.max_len = a.max_pages * c.page_size;
    if (a.prefix_len == 0) return go(own, 0, launch);

    P.prefix = 1;
    P.block_table = a.prefix_table, P.bt_stride = 0, P.lens = nullptr;
    P.requests = 1, P.rows = P.all_rows, P.max_len = a.prefix_len;
    // The dense kernel where it is the better one and its slots fit; records are always the smaller.
    const size_t slots = prefix_tc_bytes(h, c.kv_heads, P.all_rows, a.prefix_len, c.head_dim);
    const bool dense = slots && go(own, slots, false) == LQ_OK;
    const size_t pre = dense ? slots : (rows * (c.head_dim + 1) * sizeof(float) + 255) & ~size_t(255);
    if (!dense) {
        P.pre_o = reinterpret_cast<float*>(ws);
        P.pre_m = P.pre_o + rows * c.head_dim;
        const lq_status s = go(P, pre, launch);
        if (s != LQ_OK) return s;
    } else if (launch) {
        const lq_status s = launch_prefix_tc(h, P, c.bits, c.head_dim, bf16, ws, stream);
        if (s != LQ_OK) return s;
    }
    own.pre_o = P.pre_o, own.pre_m = P.pre_m;
    own.pre_rows = P.pre_rows, own.pre_tiles = P.pre_tiles, own.pre_each = P.pre_each, own.pre_total = P.pre_total;
    own.pre_blocks = P.pre_blocks, own.pre_slots = P.pre_slots;
    return go(own, pre, launch);
}

}  // namespace

lq_status launch_kv_attention(lq_handle h, const lq_kv_cache& c, const lq_kv_attention_args& a, int window, int sinks, cudaStream_t stream) {
    // all requests at once where the workspace and 32-bit indices have room for that, otherwise so many at a time that they have
    int n = a.batch;
    for (;; n = (n + 1) / 2) {
        lq_status s = attend(h, c, a, window, sinks, 0, n, false, stream);
        if (s == LQ_OK && a.batch % n) s = attend(h, c, a, window, sinks, 0, a.batch % n, false, stream);
        if (s == LQ_OK) break;
        if ((s != LQ_ERR_WORKSPACE && s != LQ_ERR_UNSUPPORTED) || n == 1) return s;
    }
    for (int first = 0; first < a.batch; first += n) {
        const lq_status s = attend(h, c, a, window, sinks, first, std::min(n, a.batch - first), true, stream);
        if (s != LQ_OK) return s;
    }
    return LQ_OK;
}

}  // namespace lq
