// What the two attention kernels share: their parameters, small device helpers, and the joining
// of a unit's partial sums.
#pragma once

#include <math.h>

#include "lq_internal.h"
#include "lq_kv.cuh"
#include "lq_share.h"
#include "lq_tma.cuh"

namespace lq {

constexpr int kMaxDevices = 64;  // devices whose kernel settings are kept
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
    int page_shift;                      // log2 of the tiles of a page, -1 when that is not whole
    float scale_log2;                    // scale * log2(e)
    float* part;                         // partial sums: 2 slots per block
    unsigned* counters;                  // one per unit, zero between calls
    // The prefix run's sums, which the second run joins with its own.  As records: normalised rows [kv_heads]
    // [rows of all requests][D] and their reference; as slots (pre_rows > 0): the prefix kernel's partial sums,
    // pre_slots slots of pre_rows rows per block, pre_blocks blocks sharing pre_total places evenly (lq_share.h).
    float *pre_o, *pre_m;
    int pre_rows, pre_tiles, pre_each, pre_total, pre_blocks, pre_slots;
    int all_rows;                        // rows of all requests per kv head
    int prefix;                          // 0: none, 1: this is the prefix run, 2: join the prefix's rows
    int* status;
    int window, sinks;                   // (attn_kernel<kWin>) a row sees its last `window` tokens and the first `sinks`
};

// n / d for a quotient below 2^20 (n, d > 0): a reciprocal and one correction.
__device__ __forceinline__ int quick_div(int n, int d) {
    int q = __float2int_rz(__fdividef((float)n, (float)d));
    const int r = n - q * d;
    return r < 0 ? q - 1 : r >= d ? q + 1 : q;
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
__device__ __forceinline__ unsigned arrive_gpu(unsigned* count) {
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
    return old;
}
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
// What the rounding of a b to p left out, exactly.
__device__ __forceinline__ uint32_t hmul2_rest(uint32_t a, uint32_t b, uint32_t p) {
    uint32_t d;
    asm("{\n\t.reg .b32 m;\n\tneg.f16x2 m, %3;\n\tfma.rn.f16x2 %0, %1, %2, m;\n\t}" : "=r"(d) : "r"(a), "r"(b), "r"(p));
    return d;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Each half all ones where a > b (not where one is NaN).
__device__ __forceinline__ uint32_t hgt2_mask(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("{\n\t.reg .pred p, q;\n\t.reg .b16 l, h;\n\tsetp.gt.f16x2 p|q, %1, %2;\n\tselp.b16 l, 0xffff, 0, p;\n\t"
        "selp.b16 h, 0xffff, 0, q;\n\tmov.b32 %0, {l, h};\n\t}"
        : "=r"(d)
        : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint32_t h) {
    return make_float2(half_bits_to_float((uint16_t)h), half_bits_to_float((uint16_t)(h >> 16)));
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <class T>
struct IsHalf {
    static constexpr bool value = false;
};
template <>
struct IsHalf<__half> {
    static constexpr bool value = true;
};

template <class T>
__device__ __forceinline__ float elem_to_float(uint16_t bits);
template <>
__device__ __forceinline__ float elem_to_float<__half>(uint16_t bits) { return half_bits_to_float(bits); }
template <>
__device__ __forceinline__ float elem_to_float<__nv_bfloat16>(uint16_t bits) { return bf16_bits_to_float(bits); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Partial sums of one row, n of them, that a warp joins: V dimensions per lane from part(k), (reference,
// sum of P) from ml(k), the first 32 in a lane's register each.  B parts' loads are in flight at a time, the
// first B from the start on.
template <int V, int B, class Part, class Ml>
struct RowParts {
    Part part;
    Ml ml;
    int n, lane;
    float2 mine;   // part `lane`'s reference and sum
    float f;       // its factor
    float o[B][V];
    __device__ __forceinline__ void load(int k0) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const float* a = part(min(k0 + j, n - 1)) + V * lane;
            if (V == 4) {
                const float4 e = __ldcg(reinterpret_cast<const float4*>(a));
                o[j][0] = e.x, o[j][1] = e.y, o[j][V - 2] = e.z, o[j][V - 1] = e.w;
            } else {
                const float2 e = __ldcg(reinterpret_cast<const float2*>(a));
                o[j][0] = e.x, o[j][1] = e.y;
            }
        }
    }
    __device__ __forceinline__ RowParts(int count, int lane_, Part p, Ml m) : part(p), ml(m), n(count), lane(lane_) {
        mine = lane < n ? ml(lane) : make_float2(-INFINITY, 0.f);
        load(0);
    }
    __device__ __forceinline__ float top() const {
        float t = mine.x;
        for (int k = 32 + lane; k < n; k += 32) t = fmaxf(t, ml(k).x);
        return warp_max(t);
    }
    // sums of P relative to `ref`
    __device__ __forceinline__ float total(float ref) {
        f = ex2(mine.x - ref);
        float l = mine.y * f;
        for (int k = 32 + lane; k < n; k += 32) {
            const float2 e = ml(k);
            l = fmaf(e.y, ex2(e.x - ref), l);
        }
        return warp_sum(l);
    }
    // v += the parts, in order
    __device__ __forceinline__ void add(float ref, float (&v)[V]) {
        for (int k0 = 0; k0 < n; k0 += B) {
            if (k0) load(k0);
            if (k0 && k0 % 32 == 0) f = k0 + lane < n ? ex2(ml(k0 + lane).x - ref) : 0.f;
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const float fj = __shfl_sync(0xffffffffu, f, (k0 + j) & 31);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (k0 + j < n) v[i] = fmaf(o[j][i], fj, v[i]);
            }
        }
    }
};
template <int V, int B, class Part, class Ml>
__device__ __forceinline__ RowParts<V, B, Part, Ml> row_parts(int n, int lane, Part p, Ml m) { return RowParts<V, B, Part, Ml>(n, lane, p, m); }

// A finished row, by one warp: V dimensions per lane in v, relative to reference m, and sum of P l.  The prefix
// run leaves a record (normalised, so its sum of P counts as 1); the second run joins the prefix's parts and
// writes out and the log-sum-exp.  row: of all requests' rows of a kv head.
template <int D, class T>
__device__ __forceinline__ void finish_row(const AttnParams& P, int row, int head, float m, float l, float (&v)[D / 32], int lane) {
    constexpr int V = D / 32;
    const int64_t rec = (int64_t)head * P.all_rows + row;
    if (P.prefix == 1) {
        const float own = l == 0.f ? 0.f : 1.f / l;
        float* o = P.pre_o + rec * D + V * lane;
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<float2*>(o + i) = make_float2(v[i] * own, v[i + 1] * own);
        if (lane == 0) P.pre_m[rec] = l == 0.f ? -INFINITY : m + log2f(l);
        return;
    }
    float top = m, total = l;
    if (P.prefix == 2) {
        auto join = [&](auto&& parts) {
            top = fmaxf(m, parts.top());
            const float ref = top == -INFINITY ? 0.f : top, own = ex2(m - ref);
            total = fmaf(l, own, parts.total(ref));
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= own;
            parts.add(ref, v);
        };
        if (P.pre_rows) {
            const int rt = row / P.pre_rows, r = row - rt * P.pre_rows, unit = head * P.pre_tiles + rt;
            const Shares shares(P.pre_total, P.pre_blocks);
            const int us = prefix_unit_place(P.pre_each, unit), c0 = shares.of(us), c1 = shares.of(us + P.pre_each - 1);
            const int slot = P.pre_rows * (D + 2), s0 = prefix_slot(shares, P.pre_each, c0, unit);
            // (every later block of the unit starts with it)
            auto at = [=](int k) { return P.pre_o + (int64_t)((c0 + k) * P.pre_slots + (k == 0 ? s0 : 0)) * slot; };
            join(row_parts<V, 8>(c1 - c0 + 1, lane, [=](int k) { return at(k) + r * D; },
                              [=](int k) { return __ldcg(reinterpret_cast<const float2*>(at(k) + (slot / (D + 2)) * D + 2 * r)); }));
        } else {
            const float *o = P.pre_o + rec * D, *pm = P.pre_m + rec;
            join(row_parts<V, 1>(1, lane, [=](int) { return o; }, [=](int) { return make_float2(__ldcg(pm), 1.f); }));
        }
    }
    const int bt = row / P.group, qh = head * P.group + (row - bt * P.group);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    alignas(4 * V) T o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = (T)(v[i] * inv);
    T* out = static_cast<T*>(P.out) + bt * P.out_stride + (int64_t)qh * D + V * lane;
    if (V == 4) *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
    else *reinterpret_cast<uint32_t*>(out) = *reinterpret_cast<const uint32_t*>(o);
    if (lane == 0 && P.lse)
        P.lse[(int64_t)bt * P.q_heads + qh] = total == 0.f ? -INFINITY : (top + log2f(total) - kPBits) * 0.6931471805599453f;
}

// A unit's partial sums of blocks c0 .. c1, joined in block order: a warp per row.
template <int D, int R, int kWarps, class T>
__device__ __forceinline__ void join(const AttnParams& P, int c0, int c1, int warp, int lane, int rows, int row0, int head) {
    constexpr int V = D / 32, kSlot = R * (D + 2);   // (slots of all blocks together: within 32 bits)
    const float* base = P.part + (unsigned)(2 * c0) * kSlot;
    for (int r = warp; r < rows; r += kWarps) {
        auto at = [=](int k) { return base + (unsigned)(2 * k + (k == 0 ? 1 : 0)) * kSlot; };
        auto parts = row_parts<V, 16>(c1 - c0 + 1, lane, [=](int k) { return at(k) + r * D; },
                                  [=](int k) { return __ldcg(reinterpret_cast<const float2*>(at(k) + R * D + 2 * r)); });
        const float top = parts.top(), ref = top == -INFINITY ? 0.f : top, l = parts.total(ref);
        float v[V] = {};
        parts.add(ref, v);
        finish_row<D, T>(P, row0 + r, head, top, l, v, lane);
    }
}

// A run's scratch, and whether it is only to be asked for (launch false).
struct Scratch {
    char* at;
    size_t room, need;
    bool launch;
    cudaStream_t stream;
};

// A run of requests through a sliding window (P.window, P.sinks).
lq_status run_attn_window(lq_handle h, AttnParams& P, int bits, int D, bool bf16, Scratch s);

// The shared prefix's run on the tensor-memory tensor cores, which leaves partial sums in `scratch`.
// prefix_tc_bytes: what it needs of that, 0 where the other kernel takes the prefix.
size_t prefix_tc_bytes(lq_handle h, int kv_heads, int all_rows, int prefix_len, int D);
lq_status launch_prefix_tc(lq_handle h, AttnParams& P, int bits, int D, bool bf16, char* scratch, cudaStream_t stream);

}  // namespace lq
