// Rotary positions and the low-bit KV cache: the rotation table, the rotation of a row (and its
// transpose), rows quantised into cache tiles as they are written, and tiles read back.
//
// All of it is bound by memory: a few operations per value, one pass over the data.  A row (one
// head of one token) is taken by D / 8 lanes, 8 values (16 bytes of a 16-bit type) each; what a
// rotation or a group's range needs of other lanes comes by shuffles, so each value is read once
// and written once.  A group of lanes stays with its token, whose cosines and sines it holds in
// registers, and walks a chunk of its rows, four loads at a time; neighbouring groups have
// neighbouring tokens, which lie in the same cache tiles.
//
// Measured (from a graph): rotation of 2048 x 40 x 128 bf16, 43 MB in 8.5 us, 5.1 TB/s; in f16, 1111 x 64 x
// 64 of which 32 rotate, strided rows, 4.0 us.  Rotation, 8-bit cache write and reading back of
// 2048 tokens, 64 query and 8 kv heads: 94 MB in 24.4 us, where the append is bound by its instructions
// (issue 66 %, 21 per value: each product and sum of a rotation is rounded by itself).

#include <math.h>
#include <string.h>

#include <algorithm>

#include "lq_internal.h"
#include "lq_kv.cuh"
#include "lq_tma.cuh"

namespace lq {
namespace {

// ---- 8 values of a row, as pairs ----------------------------------------------------------

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }

// Words of 8 values: pair i in word i (16-bit types) or in words 2 i, 2 i + 1.
template <class T>
struct Row8 {
    uint32_t w[8 * sizeof(T) / 4];

    __device__ __forceinline__ static Row8 load(const T* p) {
        Row8 r;
        *reinterpret_cast<uint4*>(r.w) = *reinterpret_cast<const uint4*>(p);
        if (sizeof(T) == 4) reinterpret_cast<uint4*>(r.w)[sizeof(T) / 4] = reinterpret_cast<const uint4*>(p)[sizeof(T) / 4];
        return r;
    }
    __device__ __forceinline__ void store(T* p) const {
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
        if (sizeof(T) == 4) reinterpret_cast<uint4*>(p)[sizeof(T) / 4] = reinterpret_cast<const uint4*>(w)[sizeof(T) / 4];
    }
    __device__ __forceinline__ float2 get(int i) const;
    __device__ __forceinline__ void set(int i, float2 v);
};
template <>
__device__ __forceinline__ float2 Row8<float>::get(int i) const { return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])); }
template <>
__device__ __forceinline__ void Row8<float>::set(int i, float2 v) { w[2 * i] = bits(v.x), w[2 * i + 1] = bits(v.y); }
template <>
__device__ __forceinline__ float2 Row8<__half>::get(int i) const {
    return make_float2(half_bits_to_float((uint16_t)w[i]), half_bits_to_float((uint16_t)(w[i] >> 16)));
}
template <>
__device__ __forceinline__ void Row8<__half>::set(int i, float2 v) { w[i] = pack_half2_rn(v.x, v.y); }
template <>
__device__ __forceinline__ float2 Row8<__nv_bfloat16>::get(int i) const {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <>
__device__ __forceinline__ void Row8<__nv_bfloat16>::set(int i, float2 v) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v.y), "f"(v.x));
}

// Two fp32 operations at a time.  (Not for a product and a sum that are to be rounded each: the assembler
// makes a packed multiplication and the addition of its product one operation, .rn or not, and the same of
// a fused operation with -0.  Scalar __fmul_rn and __fadd_rn stay two.)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return reinterpret_cast<float2&>(d);
}
// ---- rotation ---------------------------------------------------------------------------

// The rotation of the 8 dimensions 8 j .. 8 j + 7 that a lane holds: y = x c + p s with p the
// pair's other member (sign in s), products and sum rounded to fp32 each.  Half layout: pairs
// (i, i + rot / 2), the other member on the lane `src`; interleaved: pairs (2 i, 2 i + 1).
struct Turn {
    float2 c[4], s[4];
    int src;          // lane of the warp with the pairs' other members (half layout)
    bool on, inter;   // whether these dimensions turn at all
};

__device__ __forceinline__ Turn turn_for(const float* row, int j, int lane, int rot, int layout, bool inverse) {
    Turn u;
    u.inter = layout == LQ_ROPE_INTERLEAVED;
    u.on = row != nullptr && 8 * j < rot;
    u.src = lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) u.c[i] = make_float2(1.f, 1.f), u.s[i] = make_float2(0.f, 0.f);
    if (!u.on) return u;
    if (u.inter) {
        const float4 c = *reinterpret_cast<const float4*>(row + 4 * j);
        const float4 s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * j);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u.c[i] = make_float2(cc[i], cc[i]);
            u.s[i] = inverse ? make_float2(ss[i], -ss[i]) : make_float2(-ss[i], ss[i]);
        }
    } else {
        const int hv = rot / 16;             // vectors of a half
        const bool first = j < hv;
        const int i0 = 8 * (first ? j : j - hv);
        u.src = lane + (first ? hv : -hv);
        const float sign = first == inverse ? 1.f : -1.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 c = *reinterpret_cast<const float4*>(row + i0 + 4 * q);
            const float4 s = *reinterpret_cast<const float4*>(row + rot / 2 + i0 + 4 * q);
            u.c[2 * q] = make_float2(c.x, c.y), u.c[2 * q + 1] = make_float2(c.z, c.w);
            u.s[2 * q] = make_float2(sign * s.x, sign * s.y), u.s[2 * q + 1] = make_float2(sign * s.z, sign * s.w);
        }
    }
    return u;
}

// (All 32 lanes call this together.)
template <class T>
__device__ __forceinline__ Row8<T> turned(const Row8<T>& x, const Turn& u) {
    Row8<T> p = x;
    if (!u.inter) {
#pragma unroll
        for (int w = 0; w < (int)(8 * sizeof(T) / 4); ++w) p.w[w] = __shfl_sync(0xffffffffu, x.w[w], u.src);
    }
    if (!u.on) return x;
    Row8<T> y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = x.get(i), o = u.inter ? make_float2(a.y, a.x) : p.get(i);
        y.set(i, make_float2(__fadd_rn(__fmul_rn(a.x, u.c[i].x), __fmul_rn(o.x, u.s[i].x)),
                             __fadd_rn(__fmul_rn(a.y, u.c[i].y), __fmul_rn(o.y, u.s[i].y))));
    }
    return y;
}

// Row of the table for a token's position; null (and the status word's bit 2) when it has none.
__device__ __forceinline__ const float* table_row(const float* table, const int* positions, int64_t n, int rows, int rot,
                                                  int* status, bool report) {
    if (!table) return nullptr;
    const int p = positions[n];
    if (p < 0 || p >= rows) {
        if (report) atomicOr(status, kStatusIndex);
        return nullptr;
    }
    return table + (int64_t)p * rot;
}

struct RopeParams {
    const void* x;
    void* y;
    int64_t xt, xh, yt, yh;   // token and head strides in elements
    const float* table;
    const int* positions;
    int n, heads, D, rot, rows, layout, inverse;
    int lanes;                // lanes of a row: the power of two >= D / 8
    int chunk;                // rows of a token that one group of lanes takes
    int* status;
};

// blockIdx.x: 256 / lanes neighbouring tokens; blockIdx.y: a chunk of their heads.
template <class T, int U>
__global__ void __launch_bounds__(256, 4) rope_kernel(const __grid_constant__ RopeParams P) {
    pdl_launch_dependents();
    pdl_wait();
    const int j = threadIdx.x & (P.lanes - 1);
    const int64_t n = (int64_t)blockIdx.x * (256 / P.lanes) + threadIdx.x / P.lanes;
    const bool live = 8 * j < P.D && n < P.n;
    const T* x = static_cast<const T*>(P.x) + n * P.xt + 8 * j;
    T* y = static_cast<T*>(P.y) + n * P.yt + 8 * j;
    const int h0 = blockIdx.y * P.chunk, h1 = min(P.heads, h0 + P.chunk);
    Turn u;
    for (int hb = h0; hb < h1; hb += U) {   // (uniform over the block: the shuffles need all lanes)
        Row8<T> v[U] = {};
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (live && hb + k < h1) v[k] = Row8<T>::load(x + (hb + k) * P.xh);
        if (hb == h0) {                     // after the first rows' loads are on their way
            const float* row = n < P.n ? table_row(P.table, P.positions, n, P.rows, P.rot, P.status, j == 0) : nullptr;
            u = turn_for(row, j, threadIdx.x & 31, P.rot, P.layout, P.inverse != 0);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const Row8<T> r = turned(v[k], u);
            if (live && hb + k < h1) r.store(y + (hb + k) * P.yh);
        }
    }
}

// The same for any even D, rotated part, stride and alignment: one thread per pair or
// unrotated dimension.
template <class T>
__global__ void __launch_bounds__(256) rope_any_kernel(const __grid_constant__ RopeParams P) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = blockIdx.x;
    const float* row = table_row(P.table, P.positions, n, P.rows, P.rot, P.status, threadIdx.x == 0);
    const int half = P.rot / 2, each = half + P.D - P.rot;   // pairs, then single dimensions
    // (unsigned: the step past the last of almost 2^31 pairs stays a number of its own)
    for (unsigned i = blockIdx.y * 256 + threadIdx.x; i < (unsigned)(P.heads * each); i += gridDim.y * 256) {
        const int h = (int)(i / (unsigned)each), k = (int)(i - (unsigned)h * (unsigned)each);
        const T* x = static_cast<const T*>(P.x) + n * P.xt + h * P.xh;
        T* y = static_cast<T*>(P.y) + n * P.yt + h * P.yh;
        if (k >= half) {
            y[half + k] = x[half + k];
            continue;
        }
        const int a = P.layout == LQ_ROPE_INTERLEAVED ? 2 * k : k, b = P.layout == LQ_ROPE_INTERLEAVED ? 2 * k + 1 : k + half;
        const float u = to_f(x[a]), w = to_f(x[b]);
        if (!row) {
            y[a] = x[a];
            y[b] = x[b];
            continue;
        }
        const float c = row[k], s = P.inverse ? -row[half + k] : row[half + k];
        y[a] = from_f<T>(__fsub_rn(__fmul_rn(u, c), __fmul_rn(w, s)));
        y[b] = from_f<T>(__fadd_rn(__fmul_rn(w, c), __fmul_rn(u, s)));
    }
}

constexpr int kMaxRot = 256;

struct TableParams {
    uint64_t step[kMaxRot / 2];   // turns per position as 64-bit fractions
    float* out;
    int half, first, count, steps;
    float mscale;
};

// cos and sin of 2 pi frac(p u): the product wraps modulo 2^64, that is modulo one turn, exactly,
// whatever the position; of its top 32 bits (1.5e-9 radians) the rounding to fp32 keeps the angle to 9.4e-8.
__device__ __forceinline__ float2 turns(uint64_t a) {
    float s, c;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);   // (2^-31 half turns)
    return make_float2(c, s);
}

constexpr int kFine = 32, kCoarse = 16;   // positions of a step, steps of a block at most

// A position is a multiple of kFine (from the block's first) plus the rest: its angle's cosine and
// sine are the product of two unit numbers, each evaluated as above once per block.  That leaves
// one evaluation per 11 outputs and two products and two sums each, which the stores hide; direct
// evaluation was bound by its arithmetic (131072 x 128: 18.7 us, and 11.7 this way).
template <int V>
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableParams P) {
    __shared__ float2 fine[kFine][kMaxRot / 2], coarse[kCoarse][kMaxRot / 2];   // [coarse: times mscale]
    pdl_launch_dependents();
    const int half = P.half, quads = half / V;
    const int64_t r0 = (int64_t)blockIdx.x * (kFine * P.steps);
    {   // a thread keeps to one frequency (the parameters are read once)
        const int i = threadIdx.x % half, share = 256 / half;
        const uint64_t u = P.step[i];
        for (int f = threadIdx.x / half; f < kFine + P.steps; f += share) {
            if (threadIdx.x / half >= share) break;
            if (f < kFine) {
                fine[f][i] = turns((uint64_t)f * u);
            } else {
                const float2 z = turns((uint64_t)(P.first + r0 + (f - kFine) * kFine) * u);
                coarse[f - kFine][i] = make_float2(z.x * P.mscale, z.y * P.mscale);
            }
        }
    }
    __syncthreads();
    pdl_wait();   // (the rows may still be read by the kernel before)
    const int per = 256 / quads, i0 = (threadIdx.x % quads) * V;
    if ((int)threadIdx.x >= per * quads) return;
    for (int f = threadIdx.x / quads; f < kFine * P.steps; f += per) {
        const int64_t r = r0 + f;
        if (r >= P.count) break;
        alignas(16) float c[V], s[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 w = fine[f % kFine][i0 + v], z = coarse[f / kFine][i0 + v];
            c[v] = fmaf(z.x, w.x, -z.y * w.y);
            s[v] = fmaf(z.x, w.y, z.y * w.x);
        }
        float* o = P.out + r * 2 * half + i0;
        if (V == 4) {
            *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(c);
            *reinterpret_cast<float4*>(o + half) = *reinterpret_cast<const float4*>(s);
        } else {
            o[0] = c[0];
            o[half] = s[0];
        }
    }
}

// ---- the cache ----------------------------------------------------------------------------

__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// (three operands at once)
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

struct AppendParams {
    KvView cache;
    const void *q, *k, *v;
    void* q_out;
    int64_t qt, kt, vt, ot;       // token strides in elements
    const int64_t* slots;
    const float* table;
    const int* positions;
    int n, q_heads, rot, rows, layout;
    int chunk;                    // rows of a token that one group of lanes takes
    int* status;
};

// A slot's tile of head 0 and its token there; null when the cache has no such slot (reported
// when it lies past the end).
struct Place {
    uint8_t* tile;
    int64_t head_bytes;
    int tok;
};
__device__ __forceinline__ Place place_of(const KvView& c, const int64_t* slots, int64_t n, int tile_bytes, int* status, bool report) {
    const int64_t slot = slots[n];
    Place p{nullptr, (int64_t)c.tiles_per_page * tile_bytes, (int)(slot & 15)};
    const int64_t tile = slot >> 4;   // (pages are whole tiles)
    if (slot < 0 || tile >= c.num_pages * c.tiles_per_page) {
        if (slot >= 0 && report) atomicOr(status, kStatusIndex);
        return p;
    }
    const int64_t page = (tile >> 32) ? tile / c.tiles_per_page : (int64_t)((uint32_t)tile / (uint32_t)c.tiles_per_page);
    p.tile = c.pages + page * c.kv_heads * p.head_bytes + (tile - page * c.tiles_per_page) * tile_bytes;
    return p;
}

// A key or value row's group of 32 is four lanes: its range by two shuffles, its codes by the
// definition's fp32 operations (correctly rounded each, so the stored bits are one and the same
// everywhere).  blockIdx.x: neighbouring tokens; blockIdx.y: a chunk of their rows (k heads, then
// v, then q: the costlier first), the same for the whole block.
template <int BITS, int D, class T, int U>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendParams P) {
    using L = KvLayout<BITS, D>;
    constexpr int kLanes = D / 8;
    constexpr float kTop = (float)((1 << BITS) - 1);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, j = threadIdx.x % kLanes, g = j >> 2;
    const int64_t n = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    const bool live = n < P.n;
    const int hq = P.q_heads, hkv = P.cache.kv_heads, all = hq + 2 * hkv;
    const int h0 = blockIdx.y * P.chunk, h1 = min(all, h0 + P.chunk);
    Place at{nullptr, 0, 0};
    Turn u;
    for (int hb = h0; hb < h1; hb += U) {
        Row8<T> x[U] = {};
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = hb + k;
            if (live && h < h1) {
                const T* src = h < hkv       ? static_cast<const T*>(P.k) + n * P.kt + h * D
                               : h < 2 * hkv ? static_cast<const T*>(P.v) + n * P.vt + (h - hkv) * D
                                             : static_cast<const T*>(P.q) + n * P.qt + (h - 2 * hkv) * D;
                x[k] = Row8<T>::load(src + 8 * j);
            }
        }
        if (hb == h0) {   // after the first rows' loads are on their way
            const float* row = nullptr;
            if (live) {
                if (h0 < 2 * hkv) at = place_of(P.cache, P.slots, n, L::kBytes, P.status, j == 0);
                if (h0 < hkv || h1 > 2 * hkv) row = table_row(P.table, P.positions, n, P.rows, P.rot, P.status, j == 0);
            }
            u = turn_for(row, j, lane, P.rot, P.layout, false);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = hb + k;
            if (h >= h1) break;
            const bool is_v = h >= hkv && h < 2 * hkv;
            const Row8<T> y = is_v ? x[k] : turned(x[k], u);
            if (h >= 2 * hkv) {
                if (live) y.store(static_cast<T*>(P.q_out) + n * P.ot + (h - 2 * hkv) * D + 8 * j);
                continue;
            }
            float2 f[4];
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = y.get(i);
            auto range = [&] {   // of the group: four lanes
                lo = min_nan(f[0].x, f[0].y), hi = max_nan(f[0].x, f[0].y);
#pragma unroll
                for (int i = 1; i < 4; ++i) lo = min_nan(lo, f[i].x, f[i].y), hi = max_nan(hi, f[i].x, f[i].y);
#pragma unroll
                for (int s = 1; s <= 2; s <<= 1) {
                    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
                    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
                }
            };
            range();
            if (__any_sync(0xffffffffu, !(lo >= -65504.f && hi <= 65504.f))) {   // clamped only where it matters
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[i] = make_float2(max_nan(min_nan(f[i].x, 65504.f), -65504.f), max_nan(min_nan(f[i].y, 65504.f), -65504.f));
                range();
            }
            const __half S = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / kTop)), Z = __float2half_rn(lo);
            const float s = __half2float(S), z = __half2float(Z);
            // rint of the rounded quotient, without a division per value: a product with 1 / s is off
            // by at most 255 * 2^-22.4 = 4.6e-5, so it has the same nearest whole number unless it lies
            // within 1e-4 of a half.  Sums with 1.5 * 2^23 round to it and hold it in their low bits.
            constexpr float kRound = 12582912.f;
            const float inv = s > 0.f ? __fdividef(1.f, s) : 0.f;
            uint32_t c[8];
            float off = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = add2(f[i], make_float2(-z, -z)), t = fma2(d, make_float2(inv, inv), make_float2(kRound, kRound));
                const float2 e = fma2(d, make_float2(inv, inv), add2(make_float2(kRound, kRound), make_float2(-t.x, -t.y)));
                off = max_nan(off, fabsf(e.x), fabsf(e.y));
                c[2 * i] = bits(fminf(fmaxf(t.x, kRound), kRound + kTop)) & 255u;
                c[2 * i + 1] = bits(fminf(fmaxf(t.y, kRound), kRound + kTop)) & 255u;
            }
            if (!(off <= 0.4999f)) {   // close to a half, or no number
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float r = rintf(__fdiv_rn(__fsub_rn(i & 1 ? f[i >> 1].y : f[i >> 1].x, z), s));
                    c[i] = s > 0.f ? (uint32_t)fminf(fmaxf(r, 0.f), kTop) : 0u;
                }
            }
            uint32_t w[2] = {0u, 0u};   // the row's 8 codes, dimension order
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (BITS == 4) w[0] |= c[i] << (4 * i);
                else w[i >> 2] |= c[i] << (8 * (i & 3));
            }
            uint8_t* t = at.tile + (h - (is_v ? hkv : 0)) * at.head_bytes;
            const bool kept = live && at.tile != nullptr;
            const int tok = at.tok;
            if (!is_v) {
                const int ln = 4 * (tok & 7) + (j & 3), q = (tok >> 3) * L::WK + g * (L::WK / L::G);
                if (kept) {
                    if (BITS == 4) *reinterpret_cast<uint32_t*>(t + kv_word_at(ln, q)) = w[0];
                    else *reinterpret_cast<uint2*>(t + kv_word_at(ln, q)) = make_uint2(w[0], w[1]);
                    if ((j & 3) == 0) {
                        reinterpret_cast<__half*>(t + L::kKs)[tok * L::G + g] = S;
                        reinterpret_cast<__half*>(t + L::kKz)[tok * L::G + g] = Z;
                    }
                }
            } else {
                // codes of one dimension of eight (four) lanes' rows side by side
                uint32_t v0, v1 = 0;
                const int e = j / L::WV, wi = j % L::WV, jt = (tok & 1) + 2 * (tok >> 3), t4 = (tok & 7) >> 1;
                if (BITS == 4) {
                    v0 = kv_transpose_nibbles(w[0], e, L::WV);
                } else {
                    v0 = kv_transpose_bytes(w[0], e, L::WV);
                    v1 = kv_transpose_bytes(w[1], e, L::WV);
                }
                if (kept) {
                    *reinterpret_cast<uint32_t*>(t + L::kVc + kv_word_at(4 * e + t4, jt * L::WV + wi)) = v0;
                    if (BITS == 8) *reinterpret_cast<uint32_t*>(t + L::kVc + kv_word_at(4 * (e + 4) + t4, jt * L::WV + wi)) = v1;
                    if ((j & 3) == 0) {
                        reinterpret_cast<__half*>(t + L::kVs)[g * kKvTile + kv_vmeta_pos(tok)] = S;
                        reinterpret_cast<__half*>(t + L::kVz)[g * kKvTile + kv_vmeta_pos(tok)] = Z;
                    }
                }
            }
        }
    }
}

struct ReadParams {
    KvView cache;
    const int64_t* slots;
    void *k, *v;   // [n][kv_heads][D], either may be null
    int n, chunk;
    int* status;
};

// blockIdx.x: neighbouring slots; blockIdx.y: a chunk of their rows (k heads, then v).
template <int BITS, int D, class T, int U>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ ReadParams P) {
    using L = KvLayout<BITS, D>;
    constexpr int kLanes = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const int j = threadIdx.x % kLanes, g = j >> 2;
    const int64_t n = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    const bool live = n < P.n;
    const int hkv = P.cache.kv_heads, first = P.k ? 0 : hkv, all = P.v ? 2 * hkv : hkv;
    const int h0 = first + blockIdx.y * P.chunk, h1 = min(all, h0 + P.chunk);
    Place at{nullptr, 0, 0};
    if (live) at = place_of(P.cache, P.slots, n, L::kBytes, P.status, j == 0);
    const int tok = at.tok, e = j / L::WV;
    // byte of this lane's word(s) and of its group's S, for keys and for values
    const int kw = kv_word_at(4 * (tok & 7) + (j & 3), (tok >> 3) * L::WK + g * (L::WK / L::G));
    const int vw = L::kVc + kv_word_at(4 * e + ((tok & 7) >> 1), ((tok & 1) + 2 * (tok >> 3)) * L::WV + j % L::WV);
    const int km = L::kKs + 2 * (tok * L::G + g), vm = L::kVs + 2 * (g * kKvTile + kv_vmeta_pos(tok));
    for (int hb = h0; hb < h1; hb += U) {
        uint32_t w[U][2] = {};
        __half s[U] = {}, z[U] = {};
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = hb + k;
            if (at.tile && h < h1) {
                const bool is_v = h >= hkv;
                const uint8_t* t = at.tile + (h - (is_v ? hkv : 0)) * at.head_bytes;
                const uint8_t* c = t + (is_v ? vw : kw);
                w[k][0] = *reinterpret_cast<const uint32_t*>(c);
                if (BITS == 8) w[k][1] = *reinterpret_cast<const uint32_t*>(c + (is_v ? 16 * 16 : 4));   // (lane 16 further)
                const uint8_t* m = t + (is_v ? vm : km);
                s[k] = *reinterpret_cast<const __half*>(m);
                z[k] = *reinterpret_cast<const __half*>(m + L::kMeta);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = hb + k;
            if (h >= h1) break;
            const bool is_v = h >= hkv;
            if (is_v) {
                if (BITS == 4) {
                    w[k][0] = kv_transpose_nibbles(w[k][0], e, L::WV);
                } else {
                    w[k][0] = kv_transpose_bytes(w[k][0], e, L::WV);
                    w[k][1] = kv_transpose_bytes(w[k][1], e, L::WV);
                }
            }
            const float sf = __half2float(s[k]), zf = __half2float(z[k]);
            Row8<T> y;
            auto code = [&](int i) {   // 2^23 + code
                if (BITS == 8) return __uint_as_float(prmt(w[k][i >> 2], 0x4b000000u, 0x7440 + (i & 3)));
                return __uint_as_float(((w[k][0] >> (4 * i)) & 15u) | 0x4b000000u);
            };
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y.set(i, fma2(add2(make_float2(code(2 * i), code(2 * i + 1)), make_float2(-8388608.f, -8388608.f)), make_float2(sf, sf),
                              make_float2(zf, zf)));
            if (live) y.store(static_cast<T*>(is_v ? P.v : P.k) + (n * hkv + (h - (is_v ? hkv : 0))) * D + 8 * j);
        }
    }
}

// Rows that one group of lanes walks: one where all rows then still fit the device at once (about 1536
// threads an SM) and the grid's second dimension, otherwise a multiple of the four that are loaded together.
int rows_per_group(int64_t n, int lanes, int rows, int num_sms) {
    const int64_t groups = std::max<int64_t>(1, (int64_t)num_sms * 1536 / lanes);
    const int chunks = (int)std::min<int64_t>(std::min(rows, 65535), std::max<int64_t>(1, (groups + n - 1) / n));
    const int each = (rows + chunks - 1) / chunks;
    return each == 1 ? 1 : (each + 3) / 4 * 4;
}

template <class Params>
lq_status launch(void (*kernel)(Params), dim3 grid, cudaStream_t stream, const Params& P) {
    return launch_overlapped(kernel, grid, 256, 0, stream, P);
}

KvView view(const lq_kv_cache& c) {
    return KvView{static_cast<uint8_t*>(c.pages), c.num_pages, c.page_size, c.kv_heads, c.page_size / kKvTile};
}

}  // namespace

lq_status launch_rope_table(lq_handle h, const lq_rope_config& c, int first, int count, float* table, cudaStream_t stream) {
    TableParams P;
    P.out = table;
    P.half = c.rot_dim / 2;
    P.first = first;
    P.count = count;
    P.mscale = c.mscale;
    const double pi2 = 6.283185307179586;
    for (int i = 0; i < P.half; ++i) {
        const double f = pow(c.base, -2.0 * i / c.rot_dim);
        double keep = 0.0;   // share of the unscaled frequency
        if (c.original_length > 0.0) {
            const double turns = c.original_length * f / pi2;
            keep = std::min(1.0, std::max(0.0, (turns - c.low_rotations) / (c.high_rotations - c.low_rotations)));
        }
        P.step[i] = (uint64_t)nearbyint(f * (keep + (1.0 - keep) / c.factor) / pi2 * 18446744073709551616.0);
    }
    // about four blocks for every SM, which hold their tables at once
    const int64_t steps = ((int64_t)count + kFine - 1) / kFine;
    P.steps = (int)std::min<int64_t>(kCoarse, (steps + 4 * h->num_sms - 1) / (4 * h->num_sms));
    const dim3 grid((unsigned)((steps + P.steps - 1) / P.steps));
    return P.half % 4 == 0 ? launch(rope_table_kernel<4>, grid, stream, P) : launch(rope_table_kernel<1>, grid, stream, P);
}

lq_status launch_rope(lq_handle h, const lq_rope_args& a, cudaStream_t stream) {
    RopeParams P;
    P.x = a.x;
    P.y = a.y;
    P.xt = a.x_token_stride, P.xh = a.x_head_stride, P.yt = a.y_token_stride, P.yh = a.y_head_stride;
    P.table = a.table;
    P.positions = a.positions;
    P.n = a.n, P.heads = a.heads, P.D = a.head_dim, P.rot = a.rot_dim, P.rows = a.table_rows;
    P.layout = a.layout, P.inverse = a.inverse;
    P.status = h->status_flag;
    const int e = a.dtype == LQ_F32 ? 4 : 2;
    // 8 values per lane where rows and strides are 16-byte aligned and a vector turns whole;
    // otherwise one pair per thread
    const int64_t bits = (int64_t)(uintptr_t)a.x | (int64_t)(uintptr_t)a.y | P.xt * e | P.xh * e | P.yt * e | P.yh * e |
                         (int64_t)(uintptr_t)a.table;
    if (bits % 16 == 0 && P.D % 8 == 0 && P.D <= 256 && P.rot % 16 == 0) {
        P.lanes = 1;
        while (8 * P.lanes < P.D) P.lanes *= 2;
        P.chunk = rows_per_group(P.n, P.lanes, P.heads, h->num_sms);
        const int at_once = 256 / P.lanes;
        const dim3 grid((unsigned)((P.n + (int64_t)at_once - 1) / at_once), (P.heads + P.chunk - 1) / P.chunk);
        if (P.chunk > 1) {
            if (a.dtype == LQ_F32) return launch(rope_kernel<float, 4>, grid, stream, P);
            return a.dtype == LQ_F16 ? launch(rope_kernel<__half, 4>, grid, stream, P) : launch(rope_kernel<__nv_bfloat16, 4>, grid, stream, P);
        }
        if (a.dtype == LQ_F32) return launch(rope_kernel<float, 1>, grid, stream, P);
        return a.dtype == LQ_F16 ? launch(rope_kernel<__half, 1>, grid, stream, P) : launch(rope_kernel<__nv_bfloat16, 1>, grid, stream, P);
    }
    const int64_t work = (int64_t)P.heads * (P.D - P.rot / 2);
    const dim3 grid((unsigned)a.n, (unsigned)std::min<int64_t>((work + 255) / 256, 64));
    if (a.dtype == LQ_F32) return launch(rope_any_kernel<float>, grid, stream, P);
    return a.dtype == LQ_F16 ? launch(rope_any_kernel<__half>, grid, stream, P) : launch(rope_any_kernel<__nv_bfloat16>, grid, stream, P);
}

namespace {

template <int BITS, int D, int U>
lq_status append_typed(int dtype, const AppendParams& P, dim3 grid, cudaStream_t stream) {
    if (dtype == LQ_F32) return launch(kv_append_kernel<BITS, D, float, U>, grid, stream, P);
    return dtype == LQ_F16 ? launch(kv_append_kernel<BITS, D, __half, U>, grid, stream, P)
                           : launch(kv_append_kernel<BITS, D, __nv_bfloat16, U>, grid, stream, P);
}

template <int BITS, int D, int U>
lq_status read_typed(int dtype, const ReadParams& P, dim3 grid, cudaStream_t stream) {
    if (dtype == LQ_F32) return launch(kv_read_kernel<BITS, D, float, U>, grid, stream, P);
    return dtype == LQ_F16 ? launch(kv_read_kernel<BITS, D, __half, U>, grid, stream, P)
                           : launch(kv_read_kernel<BITS, D, __nv_bfloat16, U>, grid, stream, P);
}

template <int BITS, int D>
lq_status append_chunked(lq_handle h, int dtype, AppendParams& P, cudaStream_t stream) {
    constexpr int kLanes = D / 8, kAtOnce = 256 / kLanes;
    const int rows = P.q_heads + 2 * P.cache.kv_heads;
    P.chunk = rows_per_group(P.n, kLanes, rows, h->num_sms);
    const dim3 grid((unsigned)((P.n + (int64_t)kAtOnce - 1) / kAtOnce), (rows + P.chunk - 1) / P.chunk);
    return P.chunk > 1 ? append_typed<BITS, D, 4>(dtype, P, grid, stream) : append_typed<BITS, D, 1>(dtype, P, grid, stream);
}

template <int BITS, int D>
lq_status read_chunked(lq_handle h, int dtype, ReadParams& P, cudaStream_t stream) {
    constexpr int kLanes = D / 8, kAtOnce = 256 / kLanes;
    const int rows = ((P.k != nullptr) + (P.v != nullptr)) * P.cache.kv_heads;
    P.chunk = rows_per_group(P.n, kLanes, rows, h->num_sms);
    const dim3 grid((unsigned)((P.n + (int64_t)kAtOnce - 1) / kAtOnce), (rows + P.chunk - 1) / P.chunk);
    return P.chunk > 1 ? read_typed<BITS, D, 4>(dtype, P, grid, stream) : read_typed<BITS, D, 1>(dtype, P, grid, stream);
}

}  // namespace

lq_status launch_kv_append(lq_handle h, const lq_kv_cache& c, const lq_kv_append_args& a, cudaStream_t stream) {
    AppendParams P;
    P.cache = view(c);
    P.q = a.q, P.k = a.k, P.v = a.v, P.q_out = a.q_out;
    P.qt = a.q_token_stride, P.kt = a.k_token_stride, P.vt = a.v_token_stride, P.ot = a.q_out_token_stride;
    P.slots = a.slots;
    P.n = a.n;
    P.table = a.table, P.positions = a.positions;
    P.q_heads = a.q ? a.q_heads : 0, P.rot = a.rot_dim, P.rows = a.table_rows, P.layout = a.layout;
    P.status = h->status_flag;
    if (c.head_dim == 128) return c.bits == 4 ? append_chunked<4, 128>(h, a.dtype, P, stream) : append_chunked<8, 128>(h, a.dtype, P, stream);
    return c.bits == 4 ? append_chunked<4, 64>(h, a.dtype, P, stream) : append_chunked<8, 64>(h, a.dtype, P, stream);
}

lq_status launch_kv_read(lq_handle h, const lq_kv_cache& c, const int64_t* slots, int n, void* k, void* v, int dtype,
                         cudaStream_t stream) {
    ReadParams P;
    P.cache = view(c);
    P.slots = slots;
    P.n = n;
    P.k = k, P.v = v;
    P.status = h->status_flag;
    if (c.head_dim == 128) return c.bits == 4 ? read_chunked<4, 128>(h, dtype, P, stream) : read_chunked<8, 128>(h, dtype, P, stream);
    return c.bits == 4 ? read_chunked<4, 64>(h, dtype, P, stream) : read_chunked<8, 64>(h, dtype, P, stream);
}

}  // namespace lq
