// What the two attention kernels share: their parameters, small device helpers, and the joining
// of a unit's partial sums.
#pragma once

#include <math.h>

#include "lq_internal.h"
#include "lq_kv.cuh"
#include "lq_tma.cuh"

namespace lq {

constexpr float kTau = 3.f;      // a row's reference moves when a score passes it by 2^3
constexpr float kPBits = 11.f;   // P = 2^11 p

struct AttnParams {
    KvView cache;
    const void* q;
    void* out;
    float* lse;
    int64_t q_stride, out_stride, bt_stride;
    const int32_t *block_table, *lens;   // (prefix run: the prefix pages, lens null)
    int requests, rows;                  // units' outer count and rows of each per kv head
    int tokens, group, q_heads;
    int max_len, row_tiles;
    float scale_log2;                    // scale * log2(e)
    float* part;                         // partial sums: 2 slots per block
    unsigned* counters;                  // one per unit, zero between calls
    // The prefix run's sums, which the second run joins with its own.  As records: normalised rows [kv_heads]
    // [rows of all requests][D] and their reference; as slots (pre_rows > 0): the prefix kernel's partial sums,
    // two slots of pre_rows rows per block, blocks sharing pre_total key blocks evenly, pre_each per unit.
    float *pre_o, *pre_m;
    int pre_rows, pre_tiles, pre_each, pre_total, pre_blocks;
    int all_rows;                        // rows of all requests per kv head
    int prefix;                          // 0: none, 1: this is the prefix run, 2: join the prefix's rows
    int* status;
};

// n things shared out to c parties in order, the first n % c of them one more: the first of party k, and
// the party of thing i.
__device__ __forceinline__ int share_first(int n, int c, int k) { return n / c * k + min(k, n % c); }
__device__ __forceinline__ int share_of(int n, int c, int i) {
    const int q = n / c, rem = n % c;
    return i < rem * (q + 1) ? i / (q + 1) : rem + (i - rem * (q + 1)) / q;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
// m16n8k16 with binary16 operands and fp32 sums: D += A B, and D = A B.  (Not volatile: free to
// be scheduled among the mask instructions around them.)
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint32_t h) {
    return make_float2(half_bits_to_float((uint16_t)h), half_bits_to_float((uint16_t)(h >> 16)));
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <class T>
__device__ __forceinline__ float elem_to_float(uint16_t bits);
template <>
__device__ __forceinline__ float elem_to_float<__half>(uint16_t bits) { return half_bits_to_float(bits); }
template <>
__device__ __forceinline__ float elem_to_float<__nv_bfloat16>(uint16_t bits) { return bf16_bits_to_float(bits); }

// Where a row's result goes, and what joins it there: out = (v 2^(m - top) + sum of the prefix's parts) / total.
template <int D, class T>
struct RowOut {
    T* out;
    float own, top, inv;
    // the prefix's parts of this row: sums at part + k * stride (the first `lead` floats further), their
    // (reference, sum of P) the same way from ml
    const float *part, *ml;
    int64_t stride;
    int parts, lead;

    __device__ __forceinline__ const float* at(const float* p, int k) const { return p + (k == 0 ? lead : k * stride); }

    // row: of all requests' rows of a kv head; (m, l): reference and sum of P.  One lane (`writes`)
    // stores the log-sum-exp.
    __device__ __forceinline__ RowOut(const AttnParams& P, int row, int head, float m, float l, bool writes) {
        parts = 0;
        top = m;
        const int64_t rec = (int64_t)head * P.all_rows + row;
        if (P.prefix == 1) {   // a record: normalised, so its sum of P counts as 1
            own = l == 0.f ? 0.f : 1.f / l;
            inv = 1.f;
            out = reinterpret_cast<T*>(P.pre_o + rec * D);
            if (writes) P.pre_m[rec] = l == 0.f ? -INFINITY : m + log2f(l);
            return;
        }
        if (P.prefix == 2) {
            if (P.pre_rows) {
                const int rt = row / P.pre_rows, r = row - rt * P.pre_rows, us = (head * P.pre_tiles + rt) * P.pre_each;
                const int c0 = share_of(P.pre_total, P.pre_blocks, us), c1 = share_of(P.pre_total, P.pre_blocks, us + P.pre_each - 1);
                const int slot = P.pre_rows * (D + 2);
                part = P.pre_o + (int64_t)2 * c0 * slot + r * D;
                ml = P.pre_o + (int64_t)2 * c0 * slot + P.pre_rows * D + 2 * r;
                stride = 2 * slot, lead = slot, parts = c1 - c0 + 1;
            } else {
                part = P.pre_o + rec * D;
                ml = P.pre_m + rec;
                stride = 0, lead = 0, parts = 1;
            }
#pragma unroll 4
            for (int k = 0; k < parts; ++k) top = fmaxf(top, __ldcg(at(ml, k)));
        }
        const float ref = top == -INFINITY ? 0.f : top;
        own = ex2(m - ref);
        float total = l * own;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
            const float* e = at(ml, k);
            total = fmaf(P.pre_rows ? __ldcg(e + 1) : 1.f, ex2(__ldcg(e) - ref), total);
        }
        top = ref;
        inv = total == 0.f ? 0.f : 1.f / total;
        const int bt = row / P.group, qh = head * P.group + (row - bt * P.group);
        out = static_cast<T*>(P.out) + bt * P.out_stride + (int64_t)qh * D;
        if (writes && P.lse) P.lse[(int64_t)bt * P.q_heads + qh] = total == 0.f ? -INFINITY : (ref + log2f(total) - kPBits) * 0.6931471805599453f;
    }
    // V dimensions from d on
    template <int V>
    __device__ __forceinline__ void store(const AttnParams& P, int d, float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= own;
        if (P.prefix == 1) {
            float* rec = reinterpret_cast<float*>(out) + d;
            if (V == 4) *reinterpret_cast<float4*>(rec) = make_float4(v[0], v[1], v[V - 2], v[V - 1]);
            else *reinterpret_cast<float2*>(rec) = make_float2(v[0], v[1]);
            return;
        }
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
            const float f = ex2(__ldcg(at(ml, k)) - top);
            const float* o = at(part, k) + d;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 e = __ldcg(reinterpret_cast<const float2*>(o + i));
                v[i] = fmaf(e.x, f, v[i]), v[i + 1] = fmaf(e.y, f, v[i + 1]);
            }
        }
        alignas(4 * V) T o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = (T)(v[i] * inv);
        if (V == 4) *reinterpret_cast<uint2*>(out + d) = *reinterpret_cast<const uint2*>(o);
        else *reinterpret_cast<uint32_t*>(out + d) = *reinterpret_cast<const uint32_t*>(o);
    }
};

// A unit's partial sums of blocks c0 .. c1, joined in block order: a warp per row, D / 32
// dimensions per lane, the blocks' factors 32 at a time (one per lane).
template <int D, int R, int kWarps, class T>
__device__ __forceinline__ void join(const AttnParams& P, int c0, int c1, int warp, int lane, int rows, int row0, int head) {
    constexpr int V = D / 32;
    constexpr int kSlot = R * (D + 2);   // (slots of all blocks together: within 32 bits)
    auto from = [&](int k) { return P.part + (unsigned)(2 * k + (k == c0 ? 1 : 0)) * kSlot; };
    for (int r = warp; r < rows; r += kWarps) {
        float top = -INFINITY, l = 0.f, v[V] = {};
        for (int k = c0 + lane; k <= c1; k += 32) top = fmaxf(top, __ldcg(from(k) + R * D + 2 * r));
        for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float ref = top == -INFINITY ? 0.f : top;
        for (int k0 = c0; k0 <= c1; k0 += 32) {
            const int m = min(32, c1 + 1 - k0);
            float f = 0.f;
            if (lane < m) {
                const float2 e = __ldcg(reinterpret_cast<const float2*>(from(k0 + lane) + R * D + 2 * r));
                f = ex2(e.x - ref);
                l = fmaf(e.y, f, l);
            }
            // sixteen blocks' values in flight at a time
            for (int j0 = 0; j0 < m; j0 += 16) {
                float o[16][V];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float* a = from(k0 + min(j0 + j, m - 1)) + r * D + V * lane;
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float2 e = __ldcg(reinterpret_cast<const float2*>(a + i));
                        o[j][i] = e.x, o[j][i + 1] = e.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float fj = __shfl_sync(0xffffffffu, f, (j0 + j) & 31);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (j0 + j < m) v[i] = fmaf(o[j][i], fj, v[i]);
                }
            }
        }
        for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
        RowOut<D, T>(P, row0 + r, head, top, l, lane == 0).store(P, V * lane, v);
    }
}

// The shared prefix's run on the tensor-memory tensor cores, which leaves partial sums in `scratch`.
// prefix_tc_bytes: what it needs of that, 0 where the other kernel takes the prefix.
size_t prefix_tc_bytes(lq_handle h, int kv_heads, int all_rows, int prefix_len, int D);
lq_status launch_prefix_tc(lq_handle h, AttnParams& P, int bits, int D, bool bf16, char* scratch, cudaStream_t stream);

}  // namespace lq
