// Attention of a decode step over the low-bit KV cache.
//
// Bound by the cache's bytes: each key and value is read once for all rows that share its kv
// head.  Per (request, kv head) those are tokens * (q_heads / kv_heads) rows, 8 or 16 of which
// (one or two n = 8 tiles) a warp multiplies at a time with m16n8k16 binary16 MMAs, keys or
// dimensions as M, rows as N:
//   S^T [16 keys][rows]  = K  Q^T, then P = 2^(S - m), transposed in registers (movmatrix), then
//   O^T [dims][rows]    += V^T P^T.
//
// Codes become operands with one mask each.  A masked 4- or 8-bit code is a subnormal binary16,
// c * 2^-24 (or c * 2^-20 in the nibbles whose mask is 0x00f0), which the tensor cores multiply
// exactly: no conversion, no subtraction.  Scales and offsets stay out of the operands:
//   keys    q . k = sum_g S_g (q_g . c_g) + sum_g Z_g (sum of q_g): the first factor S_g comes in
//           fp32 after each group's MMAs, the second sum is one more MMA (groups as k) with the
//           group sums of q as two binary16 terms, so scores keep fp32 precision.  q is scaled
//           per row by a power of two into [2^9, 2^10) first, exact for both types.
//   values  sum_j p_j (S_gj c_j + Z_gj): P S_g as the B operand of group g's MMAs, sum p Z as one
//           more MMA (groups as M).  P = 2^11 p is rounded to binary16 (p up to 2^3 before the
//           running maximum moves), then P S 2^ks, with ks a power of two held per warp so that
//           S 2^ks stays below 3.9: the product spans 2^16 down to 2^-24, so a probability
//           keeps 11 bits down to 2^-27 of the largest.  Sums and statistics are fp32.
//
// The grid is persistent: all (request, kv head, row tile) units' 16-token tiles form one
// sequence, and block c of C takes the range [total c / C, total (c + 1) / C); its 8 warps take
// that range's tiles in turn, each with its own ring of bulk copies (a tile is one contiguous
// 1.3 .. 4.6 KB block).  A unit inside one range is finished there; a unit over several leaves
// partial sums in the workspace, and the block that arrives last joins them in block order
// (one fixed order: results repeat bit for bit).  Lengths are read on the device: no host
// synchronisation, and a captured graph serves any lengths.
//
// A shared prefix is the same kernel with every request's rows as one unit list over the prefix
// pages, run first; its normalised rows and log-sum-exps join at the end of the second run.

#include <math.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "lq_internal.h"
#include "lq_kv.cuh"
#include "lq_tma.cuh"

namespace lq {
namespace {

constexpr int kWarps = 8;
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
    float *pre_o, *pre_lse;              // the prefix's rows [kv_heads][rows of all requests][D] and log2-sum-exps
    int all_rows;                        // rows of all requests per kv head
    int prefix;                          // 0: none, 1: this is the prefix run, 2: join the prefix's rows
    int* status;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
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

template <int BITS, int D, int NT>
struct AttnSmem {
    using L = KvLayout<BITS, D>;
    static constexpr int kRows = 8 * NT;
    // ring stages per warp: what lets two blocks share an SM, 4 at most
    static constexpr int kStages = L::kBytes <= 2560 ? (NT == 1 || D == 64 ? 4 : 3) : 2;
    static constexpr int kPitch = D + 4;                                   // floats of a row of the sums
    static constexpr int kRing = 0;
    static constexpr int kRed = kRing + kWarps * kStages * L::kBytes;      // 4 x [rows][pitch] fp32
    static constexpr int kMl = kRed + 4 * kRows * kPitch * 4;              // [warps][rows] m, l
    static constexpr int kTot = kMl + kWarps * kRows * 8;                  // [rows] m, l of the unit
    static constexpr int kBars = kTot + kRows * 8;
    static constexpr int kFlags = kBars + kWarps * kStages * 8;
    static constexpr int kCum = (kFlags + kWarps * kStages * 4 + 15) / 16 * 16;   // then [requests + 1] int64
};

// The rows' sums of one warp.
template <int D, int NT>
struct State {
    float o[NT][D / 16][4];   // O^T, code part: dims (8 (2 i) + n, 8 (2 i + 1) + n) x rows (2 t, 2 t + 1), scaled
    float oz[NT][4];          // sum p Z: group n x rows
    float m[NT][2], l[NT][2];
    int ks;
};

template <int BITS, int D, int NT>
struct QFrag {
    uint32_t b[NT][D / 16][2];
    uint32_t z[NT][2];
    float f[NT][2];           // rows 2 t, 2 t + 1: 2^(-e) * scale * log2(e)
};

template <int BITS, int D, int NT, class T>
__device__ __forceinline__ void load_q(const AttnParams& P, QFrag<BITS, D, NT>& Q, int64_t row0, int rows, int head, int n, int t) {
    constexpr int G = D / 32;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + n;
        float v[G][8];
        float top = 0.f;
        if (r < rows) {
            const int64_t row = row0 + r, bt = row / P.group;
            const uint16_t* src = static_cast<const uint16_t*>(P.q) + bt * P.q_stride +
                                  (int64_t)(head * P.group + (int)(row - bt * P.group)) * D + 8 * t;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint4 u = *reinterpret_cast<const uint4*>(src + 32 * g);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[g][i] = elem_to_float<T>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
                    top = fmaxf(top, fabsf(v[g][i]));
                }
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[g][i] = 0.f;
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = top > 0.f ? 9 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
        e = min(max(e, -120), 120);
        const float up = pow2i(e), f = P.scale_log2 * pow2i(-e);
        Q.f[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);       // lane 4 n of n = 2 t
        Q.f[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[g][i] = __half2float(__float2half_rn(v[g][i] * up));
                sum += v[g][i];
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const __half h = __float2half_rn(sum), l = __float2half_rn(sum - __half2float(h));
            if (t == g >> 1) {
                hi |= (uint32_t)__half_as_ushort(h) << (16 * (g & 1));
                lo |= (uint32_t)__half_as_ushort(l) << (16 * (g & 1));
            }
            if (BITS == 4) {   // nibbles (0, 4), (1, 5) * 16 | (2, 6), (3, 7) * 16
                Q.b[nt][2 * g][0] = pack_half2_rn(v[g][0], v[g][4]);
                Q.b[nt][2 * g][1] = pack_half2_rn(v[g][1] * 0.0625f, v[g][5] * 0.0625f);
                Q.b[nt][2 * g + 1][0] = pack_half2_rn(v[g][2], v[g][6]);
                Q.b[nt][2 * g + 1][1] = pack_half2_rn(v[g][3] * 0.0625f, v[g][7] * 0.0625f);
            } else {           // bytes (0, 2), (1, 3) of two words
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    Q.b[nt][2 * g + u][0] = pack_half2_rn(v[g][4 * u], v[g][4 * u + 2]);
                    Q.b[nt][2 * g + u][1] = pack_half2_rn(v[g][4 * u + 1], v[g][4 * u + 3]);
                }
            }
        }
        Q.z[nt][0] = hi;
        Q.z[nt][1] = lo;
    }
}

// One 16-token tile in shared memory at `tile`: scores, new statistics, O.  `left`: tokens of the
// request from the tile's first on; vis: the same for each row (fewer for earlier query tokens).
template <int BITS, int D, int NT>
__device__ __forceinline__ void tile_step(uint32_t tile, const QFrag<BITS, D, NT>& Q, State<D, NT>& A, int left, bool edge,
                                          const int (&vis)[NT][2], int lane) {
    using L = KvLayout<BITS, D>;
    constexpr int G = D / 32, MT = D / 16, WK = L::WK, WV = L::WV;
    const int n = lane >> 2, t = lane & 3;

    // ---- scores ----
    float x[NT][4];
    {
        uint32_t kw[2 * WK];
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c)
            *reinterpret_cast<uint4*>(kw + 4 * c) = lds128(tile + 512 * c + 16 * lane);
        uint32_t s0[G / 2], s1[G / 2];   // S of keys n and n + 8
        if (G == 4) {
            *reinterpret_cast<uint2*>(s0) = lds64(tile + L::kKs + n * G * 2);
            *reinterpret_cast<uint2*>(s1) = lds64(tile + L::kKs + (n + 8) * G * 2);
        } else {
            s0[0] = lds32(tile + L::kKs + n * G * 2);
            s1[0] = lds32(tile + L::kKs + (n + 8) * G * 2);
        }
        uint32_t z0 = 0, z1 = 0;
        if (2 * t < G) {
            z0 = lds32(tile + L::kKz + n * G * 2 + 4 * t);
            z1 = lds32(tile + L::kKz + (n + 8) * G * 2 + 4 * t);
        }
        float tot[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[nt][i] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t a0, a1, a2, a3;
                if (BITS == 4) {
                    const uint32_t w0 = u ? kw[g] >> 8 : kw[g], w1 = u ? kw[WK + g] >> 8 : kw[WK + g];
                    a0 = w0 & 0x000f000fu, a1 = w1 & 0x000f000fu, a2 = w0 & 0x00f000f0u, a3 = w1 & 0x00f000f0u;
                } else {
                    const uint32_t w0 = kw[2 * g + u], w1 = kw[WK + 2 * g + u];
                    a0 = w0 & 0x00ff00ffu, a1 = w1 & 0x00ff00ffu, a2 = (w0 >> 8) & 0x00ff00ffu, a3 = (w1 >> 8) & 0x00ff00ffu;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt], a0, a1, a2, a3, Q.b[nt][2 * g + u][0], Q.b[nt][2 * g + u][1]);
            }
            const float2 f0 = unpack2(s0[g >> 1]), f1 = unpack2(s1[g >> 1]);
            const float sa = g & 1 ? f0.y : f0.x, sb = g & 1 ? f1.y : f1.x;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                tot[nt][0] = fmaf(sa, acc[nt][0], tot[nt][0]);
                tot[nt][1] = fmaf(sa, acc[nt][1], tot[nt][1]);
                tot[nt][2] = fmaf(sb, acc[nt][2], tot[nt][2]);
                tot[nt][3] = fmaf(sb, acc[nt][3], tot[nt][3]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float az[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(az, z0, z1, z0, z1, Q.z[nt][0], Q.z[nt][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] = fmaf(tot[nt][i], 16777216.f, az[i]) * Q.f[nt][i & 1];
            if (edge) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + 8 * (i >> 1) >= vis[nt][i & 1]) x[nt][i] = -INFINITY;
            }
        }
    }

    // ---- values' scales, and whether a row's reference or the scales' power of two has to move ----
    uint32_t vs[G][2];
    uint32_t zz[2] = {0u, 0u};
#pragma unroll
    for (int g = 0; g < G; ++g) *reinterpret_cast<uint2*>(vs[g]) = lds64(tile + L::kVs + g * 32 + 8 * t);
    if (n < G) *reinterpret_cast<uint2*>(zz) = lds64(tile + L::kVz + n * 32 + 8 * t);
    if (edge && left < kKvTile) {   // whatever lies past the request's end counts as zero
        const uint32_t k0 = (2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u);
        const uint32_t k1 = (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u);
#pragma unroll
        for (int g = 0; g < G; ++g) vs[g][0] &= k0, vs[g][1] &= k1;
        zz[0] &= k0, zz[1] &= k1;
    }
    uint32_t sc[G][2];
    auto scaled = [&] {
        const uint32_t k2 = (uint32_t)(A.ks + 15) * 0x04000400u;   // binary16 2^ks, twice
#pragma unroll
        for (int g = 0; g < G; ++g) sc[g][0] = hmul2(vs[g][0], k2), sc[g][1] = hmul2(vs[g][1], k2);
    };
    scaled();
    uint32_t big = hmax2(sc[0][0], sc[0][1]);
#pragma unroll
    for (int g = 1; g < G; ++g) big = hmax2(big, hmax2(sc[g][0], sc[g][1]));
    const float2 bf = unpack2(big);
    bool move = fmaxf(bf.x, bf.y) > 3.9f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) move |= fmaxf(x[nt][i], x[nt][i + 2]) > A.m[nt][i] + kTau;
    if (__any_sync(0xffffffffu, move)) {
        float top = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 s = unpack2(vs[g][i]);
                top = fmaxf(top, fmaxf(s.x, s.y));
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int ks = A.ks;
        if (top * pow2i(ks) > 3.9f) ks = max(-14, 127 - (int)(__float_as_uint(top) >> 23));
        const float down = pow2i(ks - A.ks);
        A.ks = ks;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float a[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = fmaxf(x[nt][i], x[nt][i + 2]);
#pragma unroll
                for (int s = 4; s <= 16; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const float now = mx > A.m[nt][i] + kTau ? mx : A.m[nt][i];
                a[i] = A.m[nt][i] == now ? 1.f : ex2(A.m[nt][i] - now);
                A.m[nt][i] = now;
                A.l[nt][i] *= a[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) A.oz[nt][i] *= a[i & 1];
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) A.o[nt][k][i] *= a[i & 1] * down;
        }
        scaled();
    }

    // ---- probabilities, transposed to the second product's operand ----
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float r0 = A.m[nt][0] == -INFINITY ? 0.f : A.m[nt][0] - kPBits, r1 = A.m[nt][1] == -INFINITY ? 0.f : A.m[nt][1] - kPBits;
        const float e0 = ex2(x[nt][0] - r0), e1 = ex2(x[nt][1] - r1), e2 = ex2(x[nt][2] - r0), e3 = ex2(x[nt][3] - r1);
        A.l[nt][0] += e0 + e2;
        A.l[nt][1] += e1 + e3;
        p[nt][0] = movmatrix(pack_half2_rn(e0, e1));
        p[nt][1] = movmatrix(pack_half2_rn(e2, e3));
        mma_f16_16816(A.oz[nt], zz[0], 0u, zz[1], 0u, p[nt][0], p[nt][1]);
    }

    // ---- O^T += V^T (P S)^T ----
    uint32_t vw[4 * WV];
#pragma unroll
    for (int c = 0; c < L::kChunks; ++c)
        *reinterpret_cast<uint4*>(vw + 4 * c) = lds128(tile + L::kVc + 512 * c + 16 * lane);
    // a slab of 8 dimensions, keys (2 t, 2 t + 1) or the same + 8
    auto slab = [&](int s, int half) -> uint32_t {
        const int wi = s % WV, e = s / WV;
        const uint32_t wa = vw[2 * half * WV + wi], wb = vw[(2 * half + 1) * WV + wi];
        if (BITS == 4) {
            const uint32_t y = prmt(wa, wb, e < 4 ? 0x5410 : 0x7632);
            const uint32_t w = (e & 2) ? y >> 8 : y;
            return w & ((e & 1) ? 0x00f000f0u : 0x000f000fu);
        }
        const uint32_t y = prmt(wa, wb, e < 2 ? 0x5410 : 0x7632);
        return ((e & 1) ? y >> 8 : y) & 0x00ff00ffu;
    };
#pragma unroll
    for (int g = 0; g < G; ++g) {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt][0] = hmul2(p[nt][0], sc[g][0]), b[nt][1] = hmul2(p[nt][1], sc[g][1]);
#pragma unroll
        for (int k = 2 * g; k < 2 * g + 2; ++k) {
            const uint32_t a0 = slab(2 * k, 0), a1 = slab(2 * k + 1, 0), a2 = slab(2 * k, 1), a3 = slab(2 * k + 1, 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(A.o[nt][k], a0, a1, a2, a3, b[nt][0], b[nt][1]);
        }
    }
}

// A finished row's element: v / l, joined with the prefix's row in the second run.
template <int D, class T>
__device__ __forceinline__ void finish(const AttnParams& P, int64_t row, int head, int d, float v, float m, float l) {
    float o = l == 0.f ? 0.f : v / l, s = l == 0.f ? -INFINITY : m + log2f(l) - kPBits;
    const int64_t at = (int64_t)head * P.all_rows + row;
    if (P.prefix == 1) {
        P.pre_o[at * D + d] = o;
        if (d == 0) P.pre_lse[at] = s;
        return;
    }
    if (P.prefix == 2) {
        const float s2 = P.pre_lse[at], top = fmaxf(s, s2);
        if (top != -INFINITY) {
            const float a = exp2f(s - top), c = exp2f(s2 - top);
            o = (o * a + P.pre_o[at * D + d] * c) / (a + c);
            s = top + log2f(a + c);
        }
    }
    const int64_t bt = row / P.group;
    const int qh = head * P.group + (int)(row - bt * P.group);
    static_cast<T*>(P.out)[bt * P.out_stride + (int64_t)qh * D + d] = (T)o;
    if (d == 0 && P.lse) P.lse[bt * P.q_heads + qh] = s * 0.6931471805599453f;
}

template <int BITS, int D, int NT, class T>
__global__ void __launch_bounds__(32 * kWarps, 2) attn_kernel(const __grid_constant__ AttnParams P) {
    using L = KvLayout<BITS, D>;
    using M = AttnSmem<BITS, D, NT>;
    constexpr int R = M::kRows, S = M::kStages, MT = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + M::kRed);
    float2* ml = reinterpret_cast<float2*>(smem + M::kMl);
    float2* total_ml = reinterpret_cast<float2*>(smem + M::kTot);
    volatile int* flags = reinterpret_cast<volatile int*>(smem + M::kFlags);
    int64_t* cum = reinterpret_cast<int64_t*>(smem + M::kCum);
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, t = lane & 3;

    // tiles of each request (one at least, so that every unit is somebody's), their running sum
    for (int b = tid; b < P.requests; b += 32 * kWarps) {
        const int len = P.lens ? min(max(__ldg(P.lens + b), 0), P.max_len) : P.max_len;
        cum[b + 1] = max(1, (len + kKvTile - 1) / kKvTile);
    }
    const uint32_t bars = smem_u32(smem + M::kBars) + 8 * S * warp;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == 0) {
        int64_t base = 0;
        for (int b0 = 0; b0 < P.requests; b0 += 32) {
            int64_t v = b0 + lane < P.requests ? cum[b0 + lane + 1] : 0;
            for (int s = 1; s < 32; s <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, v, s);
                if (lane >= s) v += o;
            }
            if (b0 + lane < P.requests) cum[b0 + lane + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) cum[0] = 0;
    }
    __syncthreads();

    // this block's range of the tile sequence; with few tiles, fewer blocks of a tile per warp
    const int per_tile = P.cache.kv_heads * P.row_tiles;   // units of a request
    const int64_t total = cum[P.requests] * per_tile;
    const int64_t C = min((int64_t)gridDim.x, (total + kWarps - 1) / kWarps);
    const int64_t c = blockIdx.x;
    if (c >= C) return;
    const int64_t g0 = total * c / C, g1 = total * (c + 1) / C;
    auto request_of = [&](int64_t gt) {   // last b with per_tile * cum[b] <= gt
        int lo = 0, hi = P.requests - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cum[mid] * per_tile <= gt) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };

    // ---- this warp's tiles: 32 addresses at a time, one per lane, issued S ahead ----
    const uint32_t ring = smem_u32(smem) + warp * S * L::kBytes;
    const int64_t mine = g1 - g0 > warp ? (g1 - g0 - warp + kWarps - 1) / kWarps : 0;
    int64_t issued = 0;
    const uint8_t* src = nullptr;
    auto issue = [&] {   // the next tile, if any, into stage issued % S
        if (issued >= mine) return;
        if ((issued & 31) == 0) {
            const int64_t gt = g0 + warp + kWarps * (issued + lane);
            src = nullptr;
            if (gt < g1) {
                const int b = request_of(gt);
                const int64_t in = gt - cum[b] * per_tile, each = cum[b + 1] - cum[b];
                const int unit = (int)(in / each), tile = (int)(in - unit * each), head = unit / P.row_tiles;
                const int len = P.lens ? min(max(__ldg(P.lens + b), 0), P.max_len) : P.max_len;
                if (tile * kKvTile < len) {
                    const int pi = tile / P.cache.tiles_per_page;
                    const int page = __ldg(P.block_table + b * P.bt_stride + pi);
                    if (page < 0 || page >= P.cache.num_pages) atomicOr(P.status, kStatusIndex);
                    else
                        src = P.cache.pages + (((int64_t)page * P.cache.kv_heads + head) * P.cache.tiles_per_page +
                                               (tile - pi * P.cache.tiles_per_page)) * (int64_t)L::kBytes;
                }
            }
        }
        if (lane == (int)(issued & 31)) {
            const int s = (int)(issued % S);
            flags[warp * S + s] = src != nullptr;
            if (src) {
                mbar_arrive_expect_tx(bars + 8 * s, L::kBytes);
                bulk_load(ring + s * L::kBytes, src, L::kBytes, bars + 8 * s);
            } else {
                mbar_arrive(bars + 8 * s);
            }
        }
        ++issued;
    };
    for (int s = 0; s < S; ++s) issue();

    int64_t done = 0;   // tiles of this warp already computed
    int own_abort = 0;
    int b = request_of(g0);
    int64_t first = cum[b] * per_tile, each = cum[b + 1] - cum[b];   // of the request: first tile, tiles per unit
    int unit = (int)((g0 - first) / each);
    for (;;) {
        const int64_t us = first + unit * each, ue = us + each;
        const int head = unit / P.row_tiles, rt = unit - head * P.row_tiles;
        const int rows = min(R, P.rows - rt * R);                    // live rows of this unit
        const int64_t row0 = (int64_t)b * P.rows + rt * R;
        const int len = P.lens ? min(max(__ldg(P.lens + b), 0), P.max_len) : P.max_len;

        QFrag<BITS, D, NT> Q;
        load_q<BITS, D, NT, T>(P, Q, row0, rows, head, n, t);
        State<D, NT> A;
        int seen[NT][2];   // tokens that rows 2 t, 2 t + 1 see
        A.ks = 15;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) A.oz[nt][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                A.m[nt][i] = -INFINITY;
                A.l[nt][i] = 0.f;
                const int r = rt * R + 8 * nt + 2 * t + i;
                seen[nt][i] = P.prefix == 1 ? len : len - P.tokens + 1 + min(r / P.group, P.tokens - 1);
            }
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) A.o[nt][k][i] = 0.f;
        }
        const int whole = P.prefix == 1 ? len : len - P.tokens + 1;   // tokens that every row sees

        const int64_t hi = min(ue, g1);
        for (; done < mine; ++done) {
            const int64_t gt = g0 + warp + kWarps * done;
            if (gt >= hi) break;
            const int s = (int)(done % S);
            mbar_wait_bounded(bars + 8 * s, (uint32_t)(done / S) & 1u, &own_abort, P.status);
            if (flags[warp * S + s]) {
                const int j0 = (int)(gt - us) * kKvTile;
                int vis[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) vis[nt][i] = seen[nt][i] - j0;
                tile_step<BITS, D, NT>(ring + s * L::kBytes, Q, A, len - j0, j0 + kKvTile > whole, vis, lane);
            }
            __syncwarp();   // all lanes have read the stage: it may be filled again
            issue();
        }

        // ---- the warps' sums of this unit joined, in warp order ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int s = 4; s <= 16; s <<= 1) A.l[nt][i] += __shfl_xor_sync(0xffffffffu, A.l[nt][i], s);
                if (n == 0) ml[warp * R + 8 * nt + 2 * t + i] = make_float2(A.m[nt][i], A.l[nt][i]);
            }
        __syncthreads();
        float fac[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * nt + 2 * t + i;
                float top = -INFINITY, l = 0.f;
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * R + r].x);
                const float ref = top == -INFINITY ? 0.f : top;
                for (int w = 0; w < kWarps; ++w) l += ml[w * R + r].y * ex2(ml[w * R + r].x - ref);
                fac[nt][i] = ex2(A.m[nt][i] - ref);
                if (warp == 0 && n == 0) total_ml[r] = make_float2(top, l);
            }
        const float up = pow2i(24 - A.ks);
        auto put = [&](bool add) {   // this warp's rows into (or onto) slot warp % 4
            float* dst = red + (warp & 3) * R * M::kPitch;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                    const float z0 = __shfl_sync(0xffffffffu, A.oz[nt][0], 4 * (k >> 1) + t);
                    const float z1 = __shfl_sync(0xffffffffu, A.oz[nt][1], 4 * (k >> 1) + t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s = 2 * k + (i >> 1);
                        const float u = BITS == 4 && (s / L::WV & 1) ? up * 0.0625f : up;
                        const float v = fmaf(A.o[nt][k][i], u, i & 1 ? z1 : z0) * fac[nt][i & 1];
                        float* at = dst + (8 * nt + 2 * t + (i & 1)) * M::kPitch + 8 * s + n;
                        *at = add ? *at + v : v;
                    }
                }
        };
        if (warp >= 4) put(false);
        __syncthreads();
        if (warp < 4) put(true);
        __syncthreads();

        const bool ends_here = ue <= g1, all_here = us >= g0 && ends_here;
        float* slot = P.part + (2 * c + (us >= g0 ? 1 : 0)) * (int64_t)(R * (D + 2));
        for (int i = tid; i < R * D; i += 32 * kWarps) {
            const int r = i / D, d = i % D;
            if (r >= rows) break;
            const float* a = red + r * M::kPitch + d;
            const float v = (a[0] + a[R * M::kPitch]) + (a[2 * R * M::kPitch] + a[3 * R * M::kPitch]);
            if (all_here) finish<D, T>(P, row0 + r, head, d, v, total_ml[r].x, total_ml[r].y);
            else slot[r * D + d] = v;
        }
        if (!all_here) {
            if (tid < rows) *reinterpret_cast<float2*>(slot + R * D + 2 * tid) = total_ml[tid];
            const int64_t c0 = ((us + 1) * C - 1) / total, c1 = (ue * C - 1) / total;   // the blocks that share the unit
            unsigned* count = P.counters + (int64_t)b * per_tile + unit;
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(count, 1u) == (unsigned)(c1 - c0);
            __syncthreads();
            if (s_last) {
                __threadfence();
                auto from = [&](int64_t k) { return P.part + (2 * k + (k == c0 ? 1 : 0)) * (int64_t)(R * (D + 2)); };
                for (int r = warp; r < rows; r += kWarps) {
                    float top = -INFINITY, l = 0.f;
                    for (int64_t k = c0 + lane; k <= c1; k += 32) top = fmaxf(top, __ldcg(from(k) + R * D + 2 * r));
                    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                    const float ref = top == -INFINITY ? 0.f : top;
                    for (int64_t k = c0 + lane; k <= c1; k += 32)
                        l += __ldcg(from(k) + R * D + 2 * r + 1) * ex2(__ldcg(from(k) + R * D + 2 * r) - ref);
                    for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
                    if (lane == 0) total_ml[r] = make_float2(top, l);
                }
                __syncthreads();
                for (int i = tid; i < rows * D; i += 32 * kWarps) {
                    const int r = i / D, d = i % D;
                    const float top = total_ml[r].x, ref = top == -INFINITY ? 0.f : top;
                    float v = 0.f;
#pragma unroll 8
                    for (int64_t k = c0; k <= c1; ++k) v = fmaf(__ldcg(from(k) + r * D + d), ex2(__ldcg(from(k) + R * D + 2 * r) - ref), v);
                    finish<D, T>(P, row0 + r, head, d, v, top, total_ml[r].y);
                }
                if (tid == 0) *count = 0;
            }
        }
        if (ue >= g1) break;
        if (++unit == per_tile) {
            unit = 0;
            ++b;
            first = cum[b] * per_tile;
            each = cum[b + 1] - cum[b];
        }
        __syncthreads();   // the sums' buffers are free again
    }
}

// Blocks of a kernel that fit on the device at once (0 on error); sets its shared-memory
// attribute, which only rises.  Kept per kernel and device.
template <int BITS, int D, int NT, class T>
int attn_blocks(int device, int num_sms, int smem) {
    struct Slot {
        int smem = 0, most = 0;
    };
    static std::mutex mu;
    static std::vector<Slot> slots;
    std::lock_guard<std::mutex> lock(mu);
    if ((int)slots.size() <= device) slots.resize(device + 1);
    Slot& s = slots[device];
    if (smem > s.most) {
        if (cudaFuncSetAttribute(attn_kernel<BITS, D, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return 0;
        s.most = smem;
    }
    static std::vector<std::pair<int, int>> known;   // (shared memory, blocks per SM), the same on every GB300
    for (const auto& k : known)
        if (k.first == smem) return k.second * num_sms;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kernel<BITS, D, NT, T>, 32 * kWarps, smem) != cudaSuccess) return 0;
    known.push_back({smem, n});
    return n * num_sms;
}

template <int BITS, int D, int NT, class T>
lq_status run(lq_handle h, AttnParams& P, char* scratch, size_t room, cudaStream_t stream) {
    constexpr int R = 8 * NT;
    P.row_tiles = (P.rows + R - 1) / R;
    const int smem = AttnSmem<BITS, D, NT>::kCum + 8 * (P.requests + 1);
    const int blocks = smem <= h->max_smem_optin ? attn_blocks<BITS, D, NT, T>(h->device, h->num_sms, smem) : 0;
    if (blocks < 1) return LQ_ERR_CUDA;
    if ((size_t)P.requests * P.cache.kv_heads * P.row_tiles > h->num_counters) return LQ_ERR_WORKSPACE;
    if ((size_t)blocks * 2 * R * (D + 2) * sizeof(float) > room) return LQ_ERR_WORKSPACE;
    P.part = reinterpret_cast<float*>(scratch);
    attn_kernel<BITS, D, NT, T><<<blocks, 32 * kWarps, smem, stream>>>(P);
    return cudaPeekAtLastError() == cudaSuccess ? LQ_OK : LQ_ERR_CUDA;
}

template <int BITS, int D>
lq_status run_typed(lq_handle h, AttnParams& P, bool bf16, char* scratch, size_t room, cudaStream_t stream) {
    // one n = 8 tile of rows where 8 hold them, two otherwise (a second tile costs a third more issue slots per key)
    if (P.rows <= 8)
        return bf16 ? run<BITS, D, 1, __nv_bfloat16>(h, P, scratch, room, stream) : run<BITS, D, 1, __half>(h, P, scratch, room, stream);
    return bf16 ? run<BITS, D, 2, __nv_bfloat16>(h, P, scratch, room, stream) : run<BITS, D, 2, __half>(h, P, scratch, room, stream);
}

}  // namespace

lq_status launch_kv_attention(lq_handle h, const lq_kv_cache& c, const lq_kv_attention_args& a, cudaStream_t stream) {
    AttnParams P;
    P.cache = KvView{static_cast<uint8_t*>(c.pages), c.num_pages, c.page_size, c.kv_heads, c.page_size / kKvTile};
    P.q = a.q, P.out = a.out, P.lse = a.lse;
    P.q_stride = a.q_token_stride, P.out_stride = a.out_token_stride;
    P.tokens = a.tokens, P.q_heads = a.q_heads, P.group = a.q_heads / c.kv_heads;
    P.scale_log2 = a.scale * 1.4426950408889634f;
    P.counters = h->counters;
    P.status = h->status_flag;
    P.all_rows = a.batch * a.tokens * P.group;
    // workspace: the prefix's rows and log-sum-exps, then partial sums
    char* ws = reinterpret_cast<char*>(h->partials);
    const size_t cap = h->partial_floats * sizeof(float), rows = (size_t)c.kv_heads * P.all_rows;
    const size_t pre = a.prefix_len > 0 ? (rows * (c.head_dim + 1) * sizeof(float) + 255) & ~size_t(255) : 0;
    if (pre > cap) return LQ_ERR_WORKSPACE;
    P.pre_o = reinterpret_cast<float*>(ws);
    P.pre_lse = P.pre_o + rows * c.head_dim;
    const bool bf16 = a.dtype == LQ_BF16;
    auto go = [&](AttnParams& p) {
        if (c.head_dim == 128)
            return c.bits == 4 ? run_typed<4, 128>(h, p, bf16, ws + pre, cap - pre, stream) : run_typed<8, 128>(h, p, bf16, ws + pre, cap - pre, stream);
        return c.bits == 4 ? run_typed<4, 64>(h, p, bf16, ws + pre, cap - pre, stream) : run_typed<8, 64>(h, p, bf16, ws + pre, cap - pre, stream);
    };
    if (a.prefix_len > 0) {
        P.prefix = 1;
        P.block_table = a.prefix_table, P.bt_stride = 0, P.lens = nullptr;
        P.requests = 1, P.rows = P.all_rows, P.max_len = a.prefix_len;
        const lq_status s = go(P);
        if (s != LQ_OK) return s;
    }
    P.prefix = a.prefix_len > 0 ? 2 : 0;
    P.block_table = a.block_table, P.bt_stride = a.block_table_stride, P.lens = a.lens;
    P.requests = a.batch, P.rows = a.tokens * P.group, P.max_len = a.max_pages * c.page_size;
    return go(P);
}

}  // namespace lq
