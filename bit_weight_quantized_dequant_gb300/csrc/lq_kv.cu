// Rotary positions and the low-bit KV cache: the rotation table, the rotation of a row (and its
// transpose), rows quantised into cache tiles as they are written, and tiles read back.
//
// All of it is bound by memory: a few operations per value, one pass over the data.  Rows are
// taken by D / 8 lanes, 8 values (16 bytes of a 16-bit type) each; what a rotation or a group's
// range needs of other lanes comes by shuffles, so each value is read once and written once.

#include <math.h>
#include <string.h>

#include <algorithm>

#include "lq_internal.h"
#include "lq_kv.cuh"

namespace lq {
namespace {

// ---- 8 values of a row ----------------------------------------------------------------

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

template <class T>
struct alignas(16) Vec8 {
    T v[8];
};

template <class T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
    Vec8<T> r;
    if (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(p);
    } else {
        reinterpret_cast<uint4*>(&r)[0] = reinterpret_cast<const uint4*>(p)[0];
        reinterpret_cast<uint4*>(&r)[sizeof(T) / 4] = reinterpret_cast<const uint4*>(p)[sizeof(T) / 4];
    }
    return r;
}
template <class T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& r) {
    if (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
    } else {
        reinterpret_cast<uint4*>(p)[0] = reinterpret_cast<const uint4*>(&r)[0];
        reinterpret_cast<uint4*>(p)[sizeof(T) / 4] = reinterpret_cast<const uint4*>(&r)[sizeof(T) / 4];
    }
}

// ---- rotation ---------------------------------------------------------------------------

// The rotation of the 8 dimensions 8 j .. 8 j + 7 that a lane holds: y = x c + p s with p the
// pair's other member (sign in s), products and sum rounded to fp32 each.  Half layout: pairs
// (i, i + rot / 2), the other member on the lane `src`; interleaved: pairs (2 i, 2 i + 1).
struct Turn {
    float c[8], s[8];
    int src;          // lane of the warp with the pairs' other members (half layout)
    bool on, inter;   // whether these dimensions turn at all
};

__device__ __forceinline__ Turn turn_for(const float* row, int j, int lane, int rot, int layout, bool inverse) {
    Turn u;
    u.inter = layout == LQ_ROPE_INTERLEAVED;
    u.on = row != nullptr && 8 * j < rot;
    u.src = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) u.c[i] = 1.f, u.s[i] = 0.f;
    if (!u.on) return u;
    if (u.inter) {
        const float4 c = *reinterpret_cast<const float4*>(row + 4 * j);
        const float4 s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * j);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u.c[2 * i] = u.c[2 * i + 1] = cc[i];
            u.s[2 * i] = inverse ? ss[i] : -ss[i];
            u.s[2 * i + 1] = inverse ? -ss[i] : ss[i];
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
            u.c[4 * q] = c.x, u.c[4 * q + 1] = c.y, u.c[4 * q + 2] = c.z, u.c[4 * q + 3] = c.w;
            u.s[4 * q] = sign * s.x, u.s[4 * q + 1] = sign * s.y, u.s[4 * q + 2] = sign * s.z, u.s[4 * q + 3] = sign * s.w;
        }
    }
    return u;
}

// (All 32 lanes call this together.)
template <class T>
__device__ __forceinline__ Vec8<T> turned(const Vec8<T>& x, const Turn& u) {
    Vec8<T> p = x;
    if (u.inter) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p.v[i] = x.v[i ^ 1];
    } else {
        constexpr int W = 8 * sizeof(T) / 4;
#pragma unroll
        for (int w = 0; w < W; ++w)
            reinterpret_cast<uint32_t*>(&p)[w] = __shfl_sync(0xffffffffu, reinterpret_cast<const uint32_t*>(&x)[w], u.src);
    }
    if (!u.on) return x;
    Vec8<T> y;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y.v[i] = from_f<T>(__fadd_rn(__fmul_rn(to_f(x.v[i]), u.c[i]), __fmul_rn(to_f(p.v[i]), u.s[i])));
    return y;
}

// Row of the table for a token's position; null (and the status word's bit 2) when it has none.
__device__ __forceinline__ const float* table_row(const float* table, const int* positions, int64_t n, int rows, int rot,
                                                  int* status) {
    if (!table) return nullptr;
    const int p = positions[n];
    if (p < 0 || p >= rows) {
        if (threadIdx.x == 0) atomicOr(status, kStatusIndex);
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
    int heads, D, rot, rows, layout, inverse;
    int lanes;                // lanes of a row: the power of two >= D / 8
    int* status;
};

// One block: one token, a chunk of its heads; each lane keeps its cos and sin for all of them.
template <class T>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams P) {
    const int64_t n = blockIdx.x;
    const int j = threadIdx.x & (P.lanes - 1), r0 = threadIdx.x / P.lanes, step = 256 / P.lanes;
    const float* row = table_row(P.table, P.positions, n, P.rows, P.rot, P.status);
    const Turn u = turn_for(row, j, threadIdx.x & 31, P.rot, P.layout, P.inverse != 0);
    const bool live = 8 * j < P.D;
    const T* x = static_cast<const T*>(P.x) + n * P.xt + 8 * j;
    T* y = static_cast<T*>(P.y) + n * P.yt + 8 * j;
    const int per = (P.heads + gridDim.y - 1) / gridDim.y, h1 = min(P.heads, (int)(blockIdx.y + 1) * per);
    for (int hb = blockIdx.y * per; hb < h1; hb += step) {   // (uniform over the block: the shuffles need all lanes)
        const int h = hb + r0;
        Vec8<T> v = {};
        if (live && h < h1) v = load8(x + h * P.xh);
        v = turned(v, u);
        if (live && h < h1) store8(y + h * P.yh, v);
    }
}

// The same for any even D, rotated part, stride and alignment: one thread per pair or
// unrotated dimension.
template <class T>
__global__ void __launch_bounds__(256) rope_any_kernel(const __grid_constant__ RopeParams P) {
    const int64_t n = blockIdx.x;
    const float* row = table_row(P.table, P.positions, n, P.rows, P.rot, P.status);
    const int half = P.rot / 2, each = half + P.D - P.rot;   // pairs, then single dimensions
    for (int i = blockIdx.y * 256 + threadIdx.x; i < P.heads * each; i += gridDim.y * 256) {
        const int h = i / each, k = i - h * each;
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
    int half, first, count;
    float mscale;
};

// cos and sin of 2 pi frac(p u): the product wraps modulo 2^64, that is modulo one turn, exactly,
// whatever the position; its top 32 bits give the angle to 1.5e-9 radians.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableParams P) {
    const int i = threadIdx.x % P.half, per = 256 / P.half;
    if ((int)threadIdx.x >= per * P.half) return;
    const uint64_t u = P.step[i];
    for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / P.half; r < P.count; r += (int64_t)gridDim.x * per) {
        const uint64_t a = (uint64_t)(P.first + r) * u;
        float s, c;
        sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);   // (2^-31 half turns)
        P.out[r * 2 * P.half + i] = c * P.mscale;
        P.out[r * 2 * P.half + P.half + i] = s * P.mscale;
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

struct AppendParams {
    KvView cache;
    const void *q, *k, *v;
    void* q_out;
    int64_t qt, kt, vt, ot;       // token strides in elements
    const int64_t* slots;
    const float* table;
    const int* positions;
    int q_heads, rot, rows, layout;
    int* status;
};

__device__ __forceinline__ uint8_t* tile_of(const KvView& c, int64_t slot, int head, int tile_bytes) {
    const int64_t page = slot / c.page_size;
    const int off = (int)(slot - page * c.page_size);
    return c.pages + ((page * c.kv_heads + head) * c.tiles_per_page + (off >> 4)) * (int64_t)tile_bytes;
}

// One block: one token, a chunk of its rows (q heads, then k, then v).  A key or value row's
// group of 32 is four lanes: its range by two shuffles, its codes by the definition's fp32
// operations (correctly rounded each, so the stored bits are one and the same everywhere).
template <int BITS, int D, class T>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendParams P) {
    using L = KvLayout<BITS, D>;
    constexpr int kLanes = D / 8, kStep = 256 / kLanes;
    constexpr float kTop = (float)((1 << BITS) - 1);
    const int64_t n = blockIdx.x;
    const int lane = threadIdx.x & 31, j = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
    const int hq = P.q_heads, hkv = P.cache.kv_heads, all = hq + 2 * hkv;
    const int64_t slot = P.slots[n], cap = P.cache.num_pages * P.cache.page_size;
    if (slot >= cap && threadIdx.x == 0) atomicOr(P.status, kStatusIndex);
    const bool kept = slot >= 0 && slot < cap;
    const float* row = table_row(P.table, P.positions, n, P.rows, P.rot, P.status);
    const Turn u = turn_for(row, j, lane, P.rot, P.layout, false);
    const int per = (all + gridDim.y - 1) / gridDim.y, h1 = min(all, (int)(blockIdx.y + 1) * per);
    const int tok = kept ? (int)(slot % P.cache.page_size) & 15 : 0;
    for (int hb = blockIdx.y * per; hb < h1; hb += kStep) {
        const int h = hb + r0;
        const bool live = h < h1, is_q = h < hq, is_v = h >= hq + hkv;
        Vec8<T> x = {};
        if (live) {
            const T* src = is_q   ? static_cast<const T*>(P.q) + n * P.qt + h * D
                           : is_v ? static_cast<const T*>(P.v) + n * P.vt + (h - hq - hkv) * D
                                  : static_cast<const T*>(P.k) + n * P.kt + (h - hq) * D;
            x = load8(src + 8 * j);
        }
        Vec8<T> y = turned(x, u);
        if (is_v) y = x;
        if (live && is_q) store8(static_cast<T*>(P.q_out) + n * P.ot + h * D + 8 * j, y);
        if (!__any_sync(0xffffffffu, live && !is_q)) continue;

        float f[8], lo, hi;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = max_nan(min_nan(to_f(y.v[i]), 65504.f), -65504.f);
            lo = i ? min_nan(lo, f[i]) : f[0];
            hi = i ? max_nan(hi, f[i]) : f[0];
        }
#pragma unroll
        for (int s = 1; s <= 2; s <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
        }
        const __half S = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / kTop)), Z = __float2half_rn(lo);
        const float s = __half2float(S), z = __half2float(Z);
        uint32_t w[2] = {0u, 0u};   // the row's 8 codes, dimension order
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t c = 0;
            if (s > 0.f) c = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(f[i], z), s)), 0.f), kTop);
            if (BITS == 4) w[0] |= c << (4 * i);
            else w[i >> 2] |= c << (8 * (i & 3));
        }
        // values: codes of one dimension of eight (four) lanes' rows side by side
        uint32_t v0, v1 = 0;
        if (BITS == 4) {
            v0 = kv_transpose_nibbles(w[0], j / L::WV, L::WV);
        } else {
            v0 = kv_transpose_bytes(w[0], j / L::WV, L::WV);
            v1 = kv_transpose_bytes(w[1], j / L::WV, L::WV);
        }
        if (!live || is_q || !kept) continue;
        const int head = is_v ? h - hq - hkv : h - hq, g = j >> 2;
        uint8_t* t = tile_of(P.cache, slot, head, L::kBytes);
        if (!is_v) {
            const int ln = 4 * (tok & 7) + (j & 3), q = (tok >> 3) * L::WK + g * (L::WK / L::G);
            if (BITS == 4) *reinterpret_cast<uint32_t*>(t + kv_word_at(ln, q)) = w[0];
            else *reinterpret_cast<uint2*>(t + kv_word_at(ln, q)) = make_uint2(w[0], w[1]);
            if ((j & 3) == 0) {
                reinterpret_cast<__half*>(t + L::kKs)[tok * L::G + g] = S;
                reinterpret_cast<__half*>(t + L::kKz)[tok * L::G + g] = Z;
            }
        } else {
            const int e = j / L::WV, wi = j % L::WV, jt = (tok & 1) + 2 * (tok >> 3), t4 = (tok & 7) >> 1;
            *reinterpret_cast<uint32_t*>(t + L::kVc + kv_word_at(4 * e + t4, jt * L::WV + wi)) = v0;
            if (BITS == 8) *reinterpret_cast<uint32_t*>(t + L::kVc + kv_word_at(4 * (e + 4) + t4, jt * L::WV + wi)) = v1;
            if ((j & 3) == 0) {
                reinterpret_cast<__half*>(t + L::kVs)[g * kKvTile + kv_vmeta_pos(tok)] = S;
                reinterpret_cast<__half*>(t + L::kVz)[g * kKvTile + kv_vmeta_pos(tok)] = Z;
            }
        }
    }
}

struct ReadParams {
    KvView cache;
    const int64_t* slots;
    void *k, *v;   // [n][kv_heads][D], either may be null
    int* status;
};

template <int BITS, int D, class T>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ ReadParams P) {
    using L = KvLayout<BITS, D>;
    constexpr int kLanes = D / 8, kStep = 256 / kLanes;
    const int64_t n = blockIdx.x;
    const int j = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes, g = j >> 2;
    const int hkv = P.cache.kv_heads, first = P.k ? 0 : hkv, all = P.v ? 2 * hkv : hkv;
    const int64_t slot = P.slots[n], cap = P.cache.num_pages * P.cache.page_size;
    if (slot >= cap && threadIdx.x == 0) atomicOr(P.status, kStatusIndex);
    const bool kept = slot >= 0 && slot < cap;
    const int tok = kept ? (int)(slot % P.cache.page_size) & 15 : 0;
    const int per = (all - first + gridDim.y - 1) / gridDim.y, h0 = first + blockIdx.y * per, h1 = min(all, h0 + per);
    for (int hb = h0; hb < h1; hb += kStep) {
        const int h = hb + r0;
        const bool live = h < h1, is_v = h >= hkv;
        const int head = is_v ? h - hkv : h;
        uint32_t w[2] = {0u, 0u};
        float s = 0.f, z = 0.f;
        if (live && kept) {
            const uint8_t* t = tile_of(P.cache, slot, head, L::kBytes);
            if (!is_v) {
                const int ln = 4 * (tok & 7) + (j & 3), q = (tok >> 3) * L::WK + g * (L::WK / L::G);
                w[0] = *reinterpret_cast<const uint32_t*>(t + kv_word_at(ln, q));
                if (BITS == 8) w[1] = *reinterpret_cast<const uint32_t*>(t + kv_word_at(ln, q + 1));
                s = __half2float(reinterpret_cast<const __half*>(t + L::kKs)[tok * L::G + g]);
                z = __half2float(reinterpret_cast<const __half*>(t + L::kKz)[tok * L::G + g]);
            } else {
                const int e = j / L::WV, wi = j % L::WV, jt = (tok & 1) + 2 * (tok >> 3), t4 = (tok & 7) >> 1;
                w[0] = *reinterpret_cast<const uint32_t*>(t + L::kVc + kv_word_at(4 * e + t4, jt * L::WV + wi));
                if (BITS == 8)
                    w[1] = *reinterpret_cast<const uint32_t*>(t + L::kVc + kv_word_at(4 * (e + 4) + t4, jt * L::WV + wi));
                s = __half2float(reinterpret_cast<const __half*>(t + L::kVs)[g * kKvTile + kv_vmeta_pos(tok)]);
                z = __half2float(reinterpret_cast<const __half*>(t + L::kVz)[g * kKvTile + kv_vmeta_pos(tok)]);
            }
        }
        uint32_t v0, v1 = 0;
        if (BITS == 4) {
            v0 = kv_transpose_nibbles(w[0], j / L::WV, L::WV);
        } else {
            v0 = kv_transpose_bytes(w[0], j / L::WV, L::WV);
            v1 = kv_transpose_bytes(w[1], j / L::WV, L::WV);
        }
        if (!live) continue;
        if (is_v) w[0] = v0, w[1] = v1;
        Vec8<T> y;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = BITS == 4 ? (w[0] >> (4 * i)) & 15u : (w[i >> 2] >> (8 * (i & 3))) & 255u;
            y.v[i] = from_f<T>(__fmaf_rn((float)c, s, z));
        }
        T* out = static_cast<T*>(is_v ? P.v : P.k) + (n * hkv + head) * D + 8 * j;
        store8(out, y);
    }
}

// Blocks of a token: its rows in as few blocks as still give every SM several.
int row_chunks(int64_t n, int rows, int rows_at_once, int num_sms) {
    const int most = (rows + rows_at_once - 1) / rows_at_once;
    return (int)std::min<int64_t>(most, std::max<int64_t>(1, (8 * (int64_t)num_sms + n - 1) / n));
}

lq_status launched() { return cudaPeekAtLastError() == cudaSuccess ? LQ_OK : LQ_ERR_CUDA; }

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
    const int per = 256 / P.half;
    const int grid = (int)std::min<int64_t>(((int64_t)count + per - 1) / per, (int64_t)h->num_sms * 32);
    rope_table_kernel<<<grid, 256, 0, stream>>>(P);
    return launched();
}

lq_status launch_rope(lq_handle h, const lq_rope_args& a, cudaStream_t stream) {
    RopeParams P;
    P.x = a.x;
    P.y = a.y;
    P.xt = a.x_token_stride, P.xh = a.x_head_stride, P.yt = a.y_token_stride, P.yh = a.y_head_stride;
    P.table = a.table;
    P.positions = a.positions;
    P.heads = a.heads, P.D = a.head_dim, P.rot = a.rot_dim, P.rows = a.table_rows;
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
        const dim3 grid((unsigned)a.n, row_chunks(a.n, P.heads, 256 / P.lanes, h->num_sms));
        if (a.dtype == LQ_F32) rope_kernel<float><<<grid, 256, 0, stream>>>(P);
        else if (a.dtype == LQ_F16) rope_kernel<__half><<<grid, 256, 0, stream>>>(P);
        else rope_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(P);
    } else {
        const int64_t work = (int64_t)P.heads * (P.D - P.rot / 2);
        const dim3 grid((unsigned)a.n, (unsigned)std::min<int64_t>((work + 255) / 256, 64));
        if (a.dtype == LQ_F32) rope_any_kernel<float><<<grid, 256, 0, stream>>>(P);
        else if (a.dtype == LQ_F16) rope_any_kernel<__half><<<grid, 256, 0, stream>>>(P);
        else rope_any_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(P);
    }
    return launched();
}

namespace {

template <int BITS, int D>
void append_typed(int dtype, const AppendParams& P, dim3 grid, cudaStream_t stream) {
    if (dtype == LQ_F32) kv_append_kernel<BITS, D, float><<<grid, 256, 0, stream>>>(P);
    else if (dtype == LQ_F16) kv_append_kernel<BITS, D, __half><<<grid, 256, 0, stream>>>(P);
    else kv_append_kernel<BITS, D, __nv_bfloat16><<<grid, 256, 0, stream>>>(P);
}

template <int BITS, int D>
void read_typed(int dtype, const ReadParams& P, dim3 grid, cudaStream_t stream) {
    if (dtype == LQ_F32) kv_read_kernel<BITS, D, float><<<grid, 256, 0, stream>>>(P);
    else if (dtype == LQ_F16) kv_read_kernel<BITS, D, __half><<<grid, 256, 0, stream>>>(P);
    else kv_read_kernel<BITS, D, __nv_bfloat16><<<grid, 256, 0, stream>>>(P);
}

}  // namespace

lq_status launch_kv_append(lq_handle h, const lq_kv_cache& c, const lq_kv_append_args& a, cudaStream_t stream) {
    AppendParams P;
    P.cache = view(c);
    P.q = a.q, P.k = a.k, P.v = a.v, P.q_out = a.q_out;
    P.qt = a.q_token_stride, P.kt = a.k_token_stride, P.vt = a.v_token_stride, P.ot = a.q_out_token_stride;
    P.slots = a.slots;
    P.table = a.table, P.positions = a.positions;
    P.q_heads = a.q ? a.q_heads : 0, P.rot = a.rot_dim, P.rows = a.table_rows, P.layout = a.layout;
    P.status = h->status_flag;
    const dim3 grid((unsigned)a.n, row_chunks(a.n, P.q_heads + 2 * c.kv_heads, 256 / (c.head_dim / 8), h->num_sms));
    if (c.head_dim == 128) c.bits == 4 ? append_typed<4, 128>(a.dtype, P, grid, stream) : append_typed<8, 128>(a.dtype, P, grid, stream);
    else c.bits == 4 ? append_typed<4, 64>(a.dtype, P, grid, stream) : append_typed<8, 64>(a.dtype, P, grid, stream);
    return launched();
}

lq_status launch_kv_read(lq_handle h, const lq_kv_cache& c, const int64_t* slots, int n, void* k, void* v, int dtype,
                         cudaStream_t stream) {
    ReadParams P;
    P.cache = view(c);
    P.slots = slots;
    P.k = k, P.v = v;
    P.status = h->status_flag;
    const int rows = ((k != nullptr) + (v != nullptr)) * c.kv_heads;
    const dim3 grid((unsigned)n, row_chunks(n, rows, 256 / (c.head_dim / 8), h->num_sms));
    if (c.head_dim == 128) c.bits == 4 ? read_typed<4, 128>(dtype, P, grid, stream) : read_typed<8, 128>(dtype, P, grid, stream);
    else c.bits == 4 ? read_typed<4, 64>(dtype, P, grid, stream) : read_typed<8, 64>(dtype, P, grid, stream);
    return launched();
}

}  // namespace lq
