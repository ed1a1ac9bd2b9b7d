// Attention of a decode step over the low-bit KV cache: the simplest form, one block per query
// row, 128 tokens at a time (a score per thread, then a dimension per thread).

#include <math.h>

#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

struct AttnParams {
    KvView cache;
    const void* q;
    void* out;
    float* lse;
    int64_t q_stride, out_stride, bt_stride;
    const int32_t *block_table, *lens, *prefix_table;
    int batch, tokens, q_heads, max_pages, prefix_len;
    float scale;
    int* status;
};

template <int BITS>
__device__ __forceinline__ float code_at(const uint8_t* region, int lane, int q, int e) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(region + kv_word_at(lane, q));
    return (float)((w >> (BITS * e)) & ((1u << BITS) - 1));
}

template <int BITS, int D>
__device__ __forceinline__ float key_at(const uint8_t* t, int tok, int d) {
    using L = KvLayout<BITS, D>;
    const int g = d / 32, r = d % 32;
    const float s = __half2float(reinterpret_cast<const __half*>(t + L::kKs)[tok * L::G + g]);
    const float z = __half2float(reinterpret_cast<const __half*>(t + L::kKz)[tok * L::G + g]);
    const int q = (tok >> 3) * L::WK + g * (L::WK / L::G) + (r % 8) / L::kPer;
    return __fmaf_rn(code_at<BITS>(t, 4 * (tok & 7) + r / 8, q, r % L::kPer), s, z);
}

template <int BITS, int D>
__device__ __forceinline__ float value_at(const uint8_t* t, int tok, int d) {
    using L = KvLayout<BITS, D>;
    const int g = d / 32, slab = d / 8, m = g * kKvTile + kv_vmeta_pos(tok);
    const float s = __half2float(reinterpret_cast<const __half*>(t + L::kVs)[m]);
    const float z = __half2float(reinterpret_cast<const __half*>(t + L::kVz)[m]);
    const int q = ((tok & 1) + 2 * (tok >> 3)) * L::WV + slab % L::WV;
    return __fmaf_rn(code_at<BITS>(t + L::kVc, 4 * (d & 7) + ((tok & 7) >> 1), q, slab / L::WV), s, z);
}

template <int BITS, int D, class T>
__global__ void __launch_bounds__(128) attn_row_kernel(const __grid_constant__ AttnParams P) {
    __shared__ float s_q[D], s_p[128], s_red[4];
    __shared__ const uint8_t* s_tile[8];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int head = h / (P.q_heads / P.cache.kv_heads), ps = P.cache.page_size;
    const int64_t row = (int64_t)b * P.tokens + t;
    if (tid < D) s_q[tid] = (float)static_cast<const T*>(P.q)[row * P.q_stride + h * D + tid];
    const int len = min(max(P.lens[b], 0), P.max_pages * ps), own = max(0, len - P.tokens + 1 + t);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int part = 0; part < 2; ++part) {
        const int n = part ? own : P.prefix_len;
        const int32_t* table = part ? P.block_table + b * P.bt_stride : P.prefix_table;
        for (int j0 = 0; j0 < n; j0 += 128) {
            __syncthreads();
            if (tid < 8) {
                const int j = j0 + 16 * tid;
                const uint8_t* tile = nullptr;
                if (j < n) {
                    const int page = table[j / ps];
                    if (page < 0 || page >= P.cache.num_pages) atomicOr(P.status, kStatusIndex);
                    else
                        tile = P.cache.pages + (((int64_t)page * P.cache.kv_heads + head) * P.cache.tiles_per_page +
                                                j % ps / 16) * (int64_t)KvLayout<BITS, D>::kBytes;
                }
                s_tile[tid] = tile;
            }
            __syncthreads();
            float x = -INFINITY;
            const uint8_t* tile = s_tile[tid >> 4];
            if (j0 + tid < n && tile) {
                x = 0.f;
                for (int d = 0; d < D; ++d) x = fmaf(s_q[d], key_at<BITS, D>(tile, tid & 15, d), x);
                x *= P.scale;
            }
            float top = x;
            for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            if ((tid & 31) == 0) s_red[tid >> 5] = top;
            __syncthreads();
            const float now = fmaxf(fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])), m);
            const float ref = now == -INFINITY ? 0.f : now, f = expf(m - ref), p = expf(x - ref);
            s_p[tid] = p;
            float sum = p;
            for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            __syncthreads();
            if ((tid & 31) == 0) s_red[tid >> 5] = sum;
            __syncthreads();
            l = l * f + ((s_red[0] + s_red[1]) + (s_red[2] + s_red[3]));
            m = now;
            if (tid < D) {
                o *= f;
                for (int j = 0; j < min(128, n - j0); ++j)
                    if (s_tile[j >> 4]) o = fmaf(s_p[j], value_at<BITS, D>(s_tile[j >> 4], j & 15, tid), o);
            }
        }
    }
    if (tid < D) static_cast<T*>(P.out)[row * P.out_stride + h * D + tid] = (T)(l == 0.f ? 0.f : o / l);
    if (tid == 0 && P.lse) P.lse[row * P.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

lq_status launch_kv_attention(lq_handle h, const lq_kv_cache& c, const lq_kv_attention_args& a, cudaStream_t stream) {
    AttnParams P;
    P.cache = KvView{static_cast<uint8_t*>(c.pages), c.num_pages, c.page_size, c.kv_heads, c.page_size / kKvTile};
    P.q = a.q, P.out = a.out, P.lse = a.lse;
    P.q_stride = a.q_token_stride, P.out_stride = a.out_token_stride, P.bt_stride = a.block_table_stride;
    P.block_table = a.block_table, P.lens = a.lens, P.prefix_table = a.prefix_table;
    P.batch = a.batch, P.tokens = a.tokens, P.q_heads = a.q_heads, P.max_pages = a.max_pages, P.prefix_len = a.prefix_len;
    P.scale = a.scale;
    P.status = h->status_flag;
    const dim3 grid(a.q_heads, a.tokens, a.batch);
    const bool bf = a.dtype == LQ_BF16;
#define LQ_ATTN(B, D) \
    bf ? attn_row_kernel<B, D, __nv_bfloat16><<<grid, 128, 0, stream>>>(P) : attn_row_kernel<B, D, __half><<<grid, 128, 0, stream>>>(P)
    if (c.head_dim == 128) {
        if (c.bits == 4) LQ_ATTN(4, 128);
        else LQ_ATTN(8, 128);
    } else {
        if (c.bits == 4) LQ_ATTN(4, 64);
        else LQ_ATTN(8, 64);
    }
#undef LQ_ATTN
    return cudaPeekAtLastError() == cudaSuccess ? LQ_OK : LQ_ERR_CUDA;
}

}  // namespace lq
