// Attention of a decode step over the low-bit KV cache: the kernel and its launch.  (Compiled twice, in lq_attn.cu and,
// for sliding windows, in lq_attn_window.cu.)
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
//           running maximum moves), then P S 2^ks, with ks held per warp and group so that
//           S 2^ks stays below 3.9: the product keeps 11 bits down to p S 2^ks = 2^-25 and is off by
//           2^-36 at least, in units of a code (S 2^ks is 2^-8 or more at the group's largest S, so for its
//           tokens 11 bits down to p = 2^-17).  Sums and statistics are fp32.
//
// The grid is persistent: all (request, kv head, row tile) units' 16-token tiles form one
// sequence, and block c of C takes the range [total c / C, total (c + 1) / C); its warps take
// that range's tiles in turn, each with its own ring of bulk copies (a tile is one contiguous
// 1.3 .. 4.6 KB block).  A unit inside one range is finished there; a unit over several leaves
// partial sums in the workspace, and the block that arrives last joins them in block order
// (one fixed order: results repeat bit for bit).  Lengths are read on the device: no host
// synchronisation, and a captured graph serves any lengths.
//
// A shared prefix runs first, with every request's rows as one unit list over the prefix pages; its
// sums join the rows' own at the end of the second run.  Few rows or a short prefix
// take this kernel for it, many rows the tensor-memory kernel (lq_attn_prefix.cu).
//
// Measured (128 dimensions, bf16): 24 requests of 1 .. 4001 tokens, 40 heads, 8 bits: 577 MB in 94 us,
// 6.1 TB/s of a copy's 6.7.  One request of 128 Ki tokens, 64 query heads over 8, 4 bits: 168 MB in 51 us,
// twice what its bytes take.  No pipe is full there (ALU 52 %, issue 53 %): 390 instructions per tile and warp in
// chains that 15 warps per SM do not cover, SMs that end unevenly (75 k to 95 k cycles of 103 k), and 3 us of start
// and 8 us from the last tile to the joined output.  333 tokens, 32 heads: 9.1 us, all latency.

#pragma once

#include <algorithm>
#include <mutex>

#include "lq_attn.cuh"

namespace lq {
namespace {

// Blocks of 8 warps, two on an SM, where units are few and long (fewer partial sums to join); of 4 warps, four
// on an SM, where there are more units than blocks, so that more of them are in flight: what a unit costs
// besides its tiles (its queries, the joining of its warps, its output) is latency.  Measured with
// 64 requests of 50 .. 200 tokens, 40 kv heads, 8 bits: 61.9 us with 8 warps, 43.9 with 4; 24 requests of 1 .. 4001 tokens, 40
// kv heads, 8 bits: 97.2 and 93.9; one request of 128 Ki tokens, 8 kv heads, 4 bits: 50.6 and 61.4.
// What a unit costs a block besides its tiles, in tiles (100 .. 4000 tokens a request, 8 kv heads, 4 bits; 28, 40 and 60
// for 8 warps: 16 requests of 16 rows 39.8, 35.6 and 35.1 us; 24 requests of 8 rows 31.1, 31.2 and 32.9):
template <int W>
constexpr int kUnitCost = W == 8 ? 40 : 20;
// Warps that share an SM's registers: 16, with 128 each.  16 rows of 128 dimensions do not fit that (600 bytes a
// thread spilled): 8, with 255.  Measured with 16 rows: 64 Ki tokens, 8 kv heads, 4 bits, 64.8 us with 16 warps and
// 40.7 with 8; in 8 bits 73.5 and 41.6.  8 rows of 128 dimensions, 16 and 8 warps: ragged batch as above 93.9 and 99.9, 64
// short requests 43.9 and 52.3, but one request of 128 Ki tokens 50.6 and 49.5 (8 bits 59.0 and 56.7).  4 rows of 64
// dimensions, 32 requests of 100 .. 16000 tokens, 4 bits: 54.6 and 72.6.
template <int D, int NT>
constexpr int kWarpsPerSm = NT == 2 && D == 128 ? 8 : 16;
constexpr int kPiece = 24;       // tiles of a piece of a unit, where one block takes one piece
// S 2^ks of a group stays at or below kMostS (2^14 times that is finite).  ks is 0 where the first tile's largest S is
// kLeastS or more, so that the multiplication is skipped; otherwise it brings the largest into [1, 2), and goes down
// when a larger one comes.  S 2^ks is exact, and P S 2^ks off by 2^-25 at most.  An S above kMostS among others
// below, as a wide value group has it (a clamped infinity: 513 in 8 bits), moves no power of two, which would cost
// every other token its bits: such products are taken one by one, in fp32.  (128 Ki tokens, 4 bits: 51 us, 347 if
// all were taken so; where all of a group's are wide together, ks is below 0 and it takes 62.)
constexpr float kMostS = 3.875f, kLeastS = 0x1p-8f;
constexpr uint32_t kMostS2 = 0x43c043c0u, kLeastS2 = 0x1c001c00u;   // (two of each in binary16)
constexpr uint32_t kUnset = 1u << 31, kNoScales = 0x0e0e0e0eu;

template <int BITS, int D, int NT, int W>
struct AttnSmem {
    using L = KvLayout<BITS, D>;
    static constexpr int kRows = 8 * NT;
    // ring stages per warp: what lets 16 warps share an SM, 4 at most (8 warps gain nothing from more)
    static constexpr int kStages = L::kBytes <= 2560 ? (NT == 1 || D == 64 ? 4 : 3) : 2;
    static constexpr int kPitch = D + 4;                                   // floats of a row of the sums
    static constexpr int kRing = 0;
    static constexpr int kRed = kRing + W * kStages * L::kBytes;           // W / 2 x [rows][pitch] fp32
    static constexpr int kMl = kRed + W / 2 * kRows * kPitch * 4;          // [warps][rows] m, l
    static constexpr int kTot = kMl + W * kRows * 8;                  // [rows] m, l of the unit
    static constexpr int kBars = kTot + kRows * 8;
    static constexpr int kCum = kBars + W * kStages * 8;              // then [requests + 1] int2
};

// The rows' sums of one warp.
template <int D, int NT>
struct State {
    float o[NT][D / 16][4];   // O^T, code part: dims (8 (2 i) + n, 8 (2 i + 1) + n) x rows (2 t, 2 t + 1), scaled
    float oz[NT][4];          // sum p Z: group n x rows
    float m[NT][2], l[NT][2]; // rows' references and sums of P
    float ref[NT][2];         // what scores lose before 2^x: m - 11, 0 while m is -inf
    uint32_t ks;              // 14 + ks of group g in bits 8 g .. 8 g + 4; kUnset before the first tile, kNoScales where all are 0
};
__device__ __forceinline__ int ks_of(uint32_t ks, int g) { return (int)(ks >> (8 * g) & 31u) - 14; }

template <int BITS, int D, int NT>
struct QFrag {
    uint32_t b[NT][D / 16][2];
    uint32_t z[NT][2];
    float f[NT][2];           // rows 2 t, 2 t + 1: 2^(-e) * scale * log2(e)
};

template <int BITS, int D, int NT, class T>
__device__ __forceinline__ void load_q(const AttnParams& P, QFrag<BITS, D, NT>& Q, int row0, int rows, int head, int n, int t) {
    constexpr int G = D / 32;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + n;
        float v[G][8];
        float top = 0.f;
        if (r < rows) {
            const int row = row0 + r, bt = row / P.group;
            const uint16_t* src = static_cast<const uint16_t*>(P.q) + bt * P.q_stride +
                                  (int64_t)(head * P.group + (row - bt * P.group)) * D + 8 * t;
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

// The powers of two of a tile's groups, and its values' scales times them in vs; the sums keep step.  Returns the tokens
// that have a wide group (S > kMostS where ks >= 0), whose scale is 0 in vs.  Seldom called, and short.
//   A group's first tile: 0, or what brings its largest S into [1, 2) where that is below kLeastS.  Below 0 only where all
//   of the group's S are wide together, within a factor that leaves S 2^ks in [kLeastS, kMostS]; at the first that is not,
//   ks is 0 from then on.  Later tiles: down, not below 0, where S 2^ks would pass kMostS.
template <int BITS, int D, int NT>
__device__ __forceinline__ uint32_t choose_scales(const uint8_t* tile, State<D, NT>& A, uint32_t k0, uint32_t k1, uint32_t (&vs)[D / 32][2], int t) {
    using L = KvLayout<BITS, D>;
    constexpr int G = D / 32;
    const uint32_t had = A.ks;
    uint32_t ks = G == 2 ? kNoScales & 0xffff0000u : 0u, wide = 0;
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        const uint2 v = lds64(tile + L::kVs + g * 32 + 8 * t);
        float S[4], most = 0.f, least = INFINITY, fit = 0.f;   // fit: the largest that is not wide
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2((i & 2 ? v.y & k1 : v.x & k0));
            S[i] = i & 1 ? f.y : f.x;
            most = fmaxf(most, S[i]);
            if (S[i] > 0.f) least = fminf(least, S[i]);
            if (S[i] <= kMostS) fit = fmaxf(fit, S[i]);
        }
#pragma unroll
        for (int s = 1; s <= 2; s <<= 1) {
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
            least = fminf(least, __shfl_xor_sync(0xffffffffu, least, s));
            fit = fmaxf(fit, __shfl_xor_sync(0xffffffffu, fit, s));
        }
        auto to_one = [](float top) { return 127 - (int)(__float_as_uint(top) >> 23); };
        int k = ks_of(had, g);
        if ((int)had < 0 && most > kMostS) k = max(to_one(most), -14);
        if (k < 0 && (most * pow2i(k) > kMostS || least * pow2i(k) < kLeastS)) k = 0;
        if (k >= 0) {
            if (k == 0 && (int)had < 0 ? fit < kLeastS : fit * pow2i(k) > kMostS) k = min(max(to_one(fit), 0), 15);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (S[i] > kMostS) wide |= 1u << (2 * t + (i & 1) + 4 * (i & 2));
        }
        ks |= (uint32_t)(k + 14) << (8 * g);
    }
    wide |= __shfl_xor_sync(0xffffffffu, wide, 1);
    wide |= __shfl_xor_sync(0xffffffffu, wide, 2);
    A.ks = ks;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint2 v = lds64(tile + L::kVs + g * 32 + 8 * t);
        const int k = ks_of(ks, g);
        vs[g][0] = v.x & k0, vs[g][1] = v.y & k1;
        if (k >= 0) vs[g][0] &= ~hgt2_mask(vs[g][0], kMostS2), vs[g][1] &= ~hgt2_mask(vs[g][1], kMostS2);
        const uint32_t k2 = (uint32_t)(k + 15) * 0x04000400u;
        vs[g][0] = hmul2(vs[g][0], k2), vs[g][1] = hmul2(vs[g][1], k2);
        const float down = pow2i(k - ks_of(had, g));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 8; ++i) A.o[nt][2 * g + (i >> 2)][i & 3] *= down;
    }
    return wide;
}

// One 16-token tile in shared memory at `tile`, its first token j0: scores, new statistics, O.
// Rows see seen[] tokens of the request's len (kEdge: some row may not see the whole tile); with kWin of those only
// the last `window` and the first `sinks`, and tokens from the first `sinks` up to `lowest` are in no row's window.
// kFine (binary16 outputs, whose own rounding is four times finer than bfloat16's): what the rounding of P S
// left out is multiplied too (error against 64 bits 4.2e-4 -> 2.7e-4 of the output at four tokens of 8
// requests, where rounding the output alone gives 2.1e-4; 20.5 -> 21.3 us).
template <int BITS, int D, int NT, bool kEdge, bool kFine, bool kWin>
__device__ __forceinline__ void tile_step(const uint8_t* tile, const QFrag<BITS, D, NT>& Q, State<D, NT>& A, int j0, int len,
                                          const int (&seen)[NT][2], int lane, int window, int sinks, int lowest) {
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
        for (int g = 0; g < G; ++g) {
            float acc[NT][4];
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
                for (int nt = 0; nt < NT; ++nt) {
                    if (u == 0) mma_first(acc[nt], a0, a1, a2, a3, Q.b[nt][2 * g][0], Q.b[nt][2 * g][1]);
                    else mma_add(acc[nt], a0, a1, a2, a3, Q.b[nt][2 * g + 1][0], Q.b[nt][2 * g + 1][1]);
                }
            }
            const float2 f0 = unpack2(s0[g >> 1]), f1 = unpack2(s1[g >> 1]);
            const float sa = g & 1 ? f0.y : f0.x, sb = g & 1 ? f1.y : f1.x;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tot[nt][i] = g ? fmaf(i < 2 ? sa : sb, acc[nt][i], tot[nt][i]) : (i < 2 ? sa : sb) * acc[nt][i];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float az[4];
            mma_first(az, z0, z1, z0, z1, Q.z[nt][0], Q.z[nt][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[nt][i] = fmaf(tot[nt][i], 16777216.f, az[i]) * Q.f[nt][i & 1];
            if (kEdge) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + n + 8 * (i >> 1);
                    if (j >= seen[nt][i & 1] || (kWin && j < seen[nt][i & 1] - window && j >= sinks)) x[nt][i] = -INFINITY;
                }
            }
        }
    }

    // ---- values' scales, and whether a row's reference or the scales' power of two has to move ----
    uint32_t vs[G][2];
    uint32_t zz[2] = {0u, 0u};
    // whatever lies past the request's end (or outside every row's window) counts as zero
    const int left = len - j0;
    auto inside = [&](int i) { return i < left && (!kWin || i >= lowest - j0 || i < sinks - j0); };
    const uint32_t k0 = (inside(2 * t) ? 0xffffu : 0u) | (inside(2 * t + 1) ? 0xffff0000u : 0u);
    const uint32_t k1 = (inside(2 * t + 8) ? 0xffffu : 0u) | (inside(2 * t + 9) ? 0xffff0000u : 0u);
    auto load_scales = [&] {
#pragma unroll
        for (int g = 0; g < G; ++g) *reinterpret_cast<uint2*>(vs[g]) = lds64(tile + L::kVs + g * 32 + 8 * t);
        if (kEdge) {
#pragma unroll
            for (int g = 0; g < G; ++g) vs[g][0] &= k0, vs[g][1] &= k1;
        }
    };
    load_scales();
    if (n < G) *reinterpret_cast<uint2*>(zz) = lds64(tile + L::kVz + n * 32 + 8 * t);
    if (kEdge) zz[0] &= k0, zz[1] &= k1;
    auto scale_by = [&](int g, int e) {
        const uint32_t k2 = (uint32_t)(e + 15) * 0x04000400u;   // binary16 2^e, twice
        vs[g][0] = hmul2(vs[g][0], k2), vs[g][1] = hmul2(vs[g][1], k2);
    };
    bool scales = false;
    if (A.ks != kNoScales) {
        __syncwarp();   // (so that this is a branch: sixteen predicated instructions for every tile took 0.9 us of 51.6)
        scales = (int)A.ks < 0;   // (kUnset)
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int k = ks_of(A.ks, g);
            scale_by(g, k);
            if (k < 0) scales |= ((hgt2_mask(kLeastS2, vs[g][0]) & hgt2_mask(vs[g][0], 0u)) | (hgt2_mask(kLeastS2, vs[g][1]) & hgt2_mask(vs[g][1], 0u))) != 0;
        }
    }
    {   // S 2^ks has to stay below kMostS so that P S stays finite
        uint32_t m = hmax2(vs[0][0], vs[0][1]);
#pragma unroll
        for (int g = 1; g < G; ++g) m = hmax2(m, hmax2(vs[g][0], vs[g][1]));
        const float2 f = unpack2(m);
        scales |= fmaxf(f.x, f.y) > kMostS;
    }
    bool move = scales;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) move |= fmaxf(x[nt][i], x[nt][i + 2]) > A.m[nt][i] + kTau;
    if (__any_sync(0xffffffffu, move)) {
        uint32_t wide = 0;   // tokens with a wide value group
        if (__any_sync(0xffffffffu, scales)) {
            // A first tile of ordinary scales, with no group's largest below kLeastS or above kMostS, needs no powers.
            uint32_t enough = (int)A.ks < 0 ? 0u : 1u << G;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float2 f = unpack2(hmax2(vs[g][0], vs[g][1]));
                enough |= (fmaxf(f.x, f.y) >= kLeastS) << g | (fmaxf(f.x, f.y) > kMostS) << G;
            }
            if (__reduce_or_sync(0xffffffffu, enough) == (1u << G) - 1u) A.ks = kNoScales;
            else wide = choose_scales<BITS, D, NT>(tile, A, kEdge ? k0 : 0xffffffffu, kEdge ? k1 : 0xffffffffu, vs, t);
        }
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
                A.ref[nt][i] = now == -INFINITY ? 0.f : now - kPBits;
                A.l[nt][i] *= a[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) A.oz[nt][i] *= a[i & 1];
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) A.o[nt][k][i] *= a[i & 1];
        }
        if (wide) {   // seldom: the products of these tokens' wide groups one by one, in fp32, in the units of the sums
#pragma unroll 1
            for (uint32_t rest = wide; rest; rest &= rest - 1) {
                const int j = __ffs((int)rest) - 1;
                float f[NT][2];   // P of rows 2 t, 2 t + 1, rounded as it is against Z: the two parts of a value cancel where it is small
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        f[nt][i] = __half2float(__float2half_rn(__shfl_sync(0xffffffffu, ex2((j & 8 ? x[nt][i + 2] : x[nt][i]) - A.ref[nt][i]), 4 * (j & 7) + t)));
                uint32_t w[WV];
#pragma unroll
                for (int i = 0; i < WV; ++i) w[i] = lds32(tile + L::kVc + kv_word_at(4 * n + ((j & 7) >> 1), ((j & 1) + 2 * (j >> 3)) * WV + i));
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float S = __half2float(*reinterpret_cast<const __half*>(tile + L::kVs + 2 * (g * kKvTile + kv_vmeta_pos(j))));
                    if (!(S > kMostS) || ks_of(A.ks, g) < 0) continue;
                    const float u = S * pow2i(ks_of(A.ks, g) - 24);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int k = 2 * g + (i >> 2), s = 2 * k + (i >> 1 & 1);
                            const uint32_t c = (w[s % WV] >> (BITS * (s / WV))) & ((1u << BITS) - 1u);
                            const float fu = f[nt][i & 1] == 0.f ? 0.f : f[nt][i & 1] * (BITS == 4 && (s / WV & 1) ? 16.f * u : u);
                            A.o[nt][k][i & 3] = fmaf((float)c, fu, A.o[nt][k][i & 3]);
                        }
                }
            }
        }
    }

    // A NaN or infinity of a value is for the rows that see its token.  P is 0 in the others, but 0 times it is not: P S
    // is cleared there, and a Z that is no number leaves the sums' operand and makes S one instead, which stays in
    // its group of dimensions as Z does.
    uint32_t row_sees[NT][2];
    if (kEdge) {
        auto odd = [](uint32_t z, int h) { return (z >> (16 * h) & 0x7c00u) == 0x7c00u; };
        const bool any_odd = odd(zz[0], 0) || odd(zz[0], 1) || odd(zz[1], 0) || odd(zz[1], 1);
        if (__any_sync(0xffffffffu, any_odd)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = q >> 1, shift = 16 * (q & 1);
                const uint32_t m = __ballot_sync(0xffffffffu, odd(zz[i], q & 1));   // bit 4 g + t: group g, this lane's token q
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (m >> (4 * g + t) & 1u) vs[g][i] |= 0x7fffu << shift;
                if (odd(zz[i], q & 1)) zz[i] &= ~(0xffffu << shift);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {   // (row n's count lies in lane n / 2)
            const int even = __shfl_sync(0xffffffffu, seen[nt][0], n >> 1), other = __shfl_sync(0xffffffffu, seen[nt][1], n >> 1);
            const int sees = (n & 1 ? other : even) - j0;
            auto in_view = [&](int i) { return i < sees && (!kWin || i >= sees - window || i < sinks - j0); };
            row_sees[nt][0] = (in_view(2 * t) ? 0xffffu : 0u) | (in_view(2 * t + 1) ? 0xffff0000u : 0u);
            row_sees[nt][1] = (in_view(2 * t + 8) ? 0xffffu : 0u) | (in_view(2 * t + 9) ? 0xffff0000u : 0u);
        }
    }

    // ---- probabilities, transposed to the second product's operand ----
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float e0 = ex2(x[nt][0] - A.ref[nt][0]), e1 = ex2(x[nt][1] - A.ref[nt][1]);
        const float e2 = ex2(x[nt][2] - A.ref[nt][0]), e3 = ex2(x[nt][3] - A.ref[nt][1]);
        A.l[nt][0] += e0 + e2;
        A.l[nt][1] += e1 + e3;
        p[nt][0] = movmatrix(pack_half2_rn(e0, e1));
        p[nt][1] = movmatrix(pack_half2_rn(e2, e3));
        mma_add(A.oz[nt], zz[0], 0u, zz[1], 0u, p[nt][0], p[nt][1]);
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
        uint32_t b[NT][2], rest[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                b[nt][i] = hmul2(p[nt][i], vs[g][i]);
                if (kFine) rest[nt][i] = hmul2_rest(p[nt][i], vs[g][i], b[nt][i]);
                if (kEdge) b[nt][i] &= row_sees[nt][i];
                if (kEdge && kFine) rest[nt][i] &= row_sees[nt][i];
            }
#pragma unroll
        for (int k = 2 * g; k < 2 * g + 2; ++k) {
            const uint32_t a0 = slab(2 * k, 0), a1 = slab(2 * k + 1, 0), a2 = slab(2 * k, 1), a3 = slab(2 * k + 1, 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_add(A.o[nt][k], a0, a1, a2, a3, b[nt][0], b[nt][1]);
                if (kFine) mma_add(A.o[nt][k], a0, a1, a2, a3, rest[nt][0], rest[nt][1]);
            }
        }
    }
}

// kWin: a sliding window.  A request's sequence of tiles is then those of the sinks and those from the first row's window
// on; the tiles between are neither counted nor read.  32 requests of 100 .. 5001 tokens, 40 heads, 8 bits, a window of 1024 and
// 16 sinks: 346 MB in 70 us, 4.9 TB/s; the last 4096 of 128 Ki tokens and 4 sinks, 64 heads over 8, 4 bits: 12.7 us, latency (51 for
// all of them).  A variant of its own, so that its bounds cost the others nothing.
template <int BITS, int D, int NT, int W, class T, bool kWin>
__global__ void __launch_bounds__(32 * W, kWarpsPerSm<D, NT> / W) attn_kernel(const __grid_constant__ AttnParams P) {
    using L = KvLayout<BITS, D>;
    using M = AttnSmem<BITS, D, NT, W>;
    constexpr int kCost = kUnitCost<W>;
    constexpr int R = M::kRows, S = M::kStages, MT = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + M::kRed);
    float2* ml = reinterpret_cast<float2*>(smem + M::kMl);
    float2* total_ml = reinterpret_cast<float2*>(smem + M::kTot);
    int2* cum = reinterpret_cast<int2*>(smem + M::kCum);   // running sums over requests of a unit's (tiles, pieces)
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, t = lane & 3;

    const uint32_t bars = smem_u32(smem + M::kBars) + 8 * S * warp;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    auto len_of = [&](int b) { return P.lens ? min(max(P.lens[b], 0), P.max_len) : P.max_len; };
    // tiles of a request of `len` tokens that hold sinks only, and those left out between them and the windows
    auto gap_of = [&](int len) {
        const int from = kWin ? max(0, len - P.tokens - P.window + 1) / kKvTile : 0;
        const int sunk = kWin ? min((P.sinks + kKvTile - 1) / kKvTile, from) : 0;
        return make_int2(sunk, from - sunk);
    };
    // a unit has one tile at least, so that every unit is somebody's
    for (int b = tid; b < P.requests; b += 32 * W) {
        const int tiles = max(1, (len_of(b) + kKvTile - 1) / kKvTile - gap_of(len_of(b)).y);
        cum[b + 1] = make_int2(tiles, (tiles + kPiece - 1) / kPiece);
    }
    __syncthreads();
    if (warp == 0) {
        int2 base = make_int2(0, 0);
        for (int b0 = 0; b0 < P.requests; b0 += 32) {
            int2 v = b0 + lane < P.requests ? cum[b0 + lane + 1] : make_int2(0, 0);
            for (int s = 1; s < 32; s <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, v.x, s), y = __shfl_up_sync(0xffffffffu, v.y, s);
                if (lane >= s) v.x += x, v.y += y;
            }
            if (b0 + lane < P.requests) cum[b0 + lane + 1] = make_int2(base.x + v.x, base.y + v.y);
            base.x += __shfl_sync(0xffffffffu, v.x, 31);
            base.y += __shfl_sync(0xffffffffu, v.y, 31);
        }
        if (lane == 0) cum[0] = make_int2(0, 0);
    }
    __syncthreads();

    // This block's tiles [g0, g1) of the sequence: a piece of one unit where all pieces fit the grid at once,
    // an equal share of all tiles otherwise.
    const int per = P.cache.kv_heads * P.row_tiles;   // units of a request
    const int c = blockIdx.x, C = gridDim.x;
    const bool pieces = (int64_t)cum[P.requests].y * per <= C;
    // (a share counts kCost tiles before each unit's own, for what a unit costs a block besides them)
    const int total = (cum[P.requests].x + kCost * P.requests) * per;
    const Shares shares(total, C);
    // last request b with per * start(b) <= at: for the warp together, and for each lane its own
    auto last = [&](auto start, int at) {
        int lo = 0;
        for (int step = P.requests > 32 ? 32 : 1; step; step = step == 32 ? 1 : 0) {
            const int i = lo + step * lane;
            const uint32_t in = __ballot_sync(0xffffffffu, i < P.requests && start(min(i, P.requests - 1)) * per <= at);
            lo += step * (31 - __clz((int)in));
        }
        return lo;
    };
    auto last_lane = [&](auto start, int at) {
        int lo = 0, hi = P.requests - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start(mid) * per <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    auto tiles_to = [&](int i) { return cum[i].x; };
    auto costly = [&](int i) { return cum[i].x + kCost * i; };
    auto tile_at = [&](int at) {                      // first tile at or after a place of the shares' sequence
        if (at >= total) return cum[P.requests].x * per;
        const int i = last(costly, at), tiles = cum[i + 1].x - cum[i].x, in = at - costly(i) * per;
        const int u = quick_div(in, tiles + kCost);
        return cum[i].x * per + u * tiles + max(0, in - u * (tiles + kCost) - kCost);
    };
    int g0, g1, b, unit, piece = 0, of = 1;
    if (pieces) {
        if (c >= cum[P.requests].y * per) return;
        b = last([&](int i) { return cum[i].y; }, c);
        of = cum[b + 1].y - cum[b].y;
        unit = quick_div(c - cum[b].y * per, of);
        piece = c - cum[b].y * per - unit * of;
        const int each = cum[b + 1].x - cum[b].x, us = cum[b].x * per + unit * each;
        const int pq = quick_div(each, of), pr = each - pq * of;
        g0 = us + pq * piece + min(piece, pr);
        g1 = us + pq * (piece + 1) + min(piece + 1, pr);
    } else {
        g0 = tile_at(shares.first(c));
        g1 = tile_at(shares.first(c + 1));
        if (g0 >= g1) return;
        b = last(tiles_to, g0);
        unit = quick_div(g0 - cum[b].x * per, cum[b + 1].x - cum[b].x);
    }

    // ---- this warp's tiles: 32 addresses at a time, one per lane, issued S ahead ----
    const uint32_t ring = smem_u32(smem) + warp * S * L::kBytes;
    const int mine = g1 - g0 > warp ? (g1 - g0 - warp + W - 1) / W : 0;
    int issued = 0, is = 0;               // tiles issued, the stage of the next
    uint32_t known = 0, there = 0;        // bit per lane: tile in the cache; bit per stage: the same
    const uint8_t* src = nullptr;
    auto issue = [&] {
        if (issued >= mine) return;
        const int who = issued & 31;
        if (who == 0) {
            const int gt = g0 + warp + W * (issued + lane);
            src = nullptr;
            if (gt < g1) {
                const int bb = pieces ? b : last_lane(tiles_to, gt);
                const int in = gt - cum[bb].x * per, each = cum[bb + 1].x - cum[bb].x;
                const int u = quick_div(in, each), head = P.row_tiles == 1 ? u : u / P.row_tiles;
                int tile = in - u * each;
                if (kWin) {
                    const int2 gap = gap_of(len_of(bb));
                    if (tile >= gap.x) tile += gap.y;
                }
                if (tile * kKvTile < len_of(bb)) {
                    const int pi = P.page_shift >= 0 ? tile >> P.page_shift : tile / P.cache.tiles_per_page;
                    const int page = P.block_table[bb * P.bt_stride + pi];
                    if (page < 0 || page >= P.cache.num_pages) atomicOr(P.status, kStatusIndex);
                    else
                        src = P.cache.pages + (((int64_t)page * P.cache.kv_heads + head) * P.cache.tiles_per_page +
                                               (tile - pi * P.cache.tiles_per_page)) * (int64_t)L::kBytes;
                }
            }
            known = __ballot_sync(0xffffffffu, src != nullptr);
        }
        if (lane == who) {
            if (src) {
                mbar_arrive_expect_tx(bars + 8 * is, L::kBytes);
                bulk_load(ring + is * L::kBytes, src, L::kBytes, bars + 8 * is);
            } else {
                mbar_arrive(bars + 8 * is);
            }
        }
        there = (there & ~(1u << is)) | ((known >> who & 1u) << is);
        is = is + 1 == S ? 0 : is + 1;
        ++issued;
    };
#pragma unroll 1
    for (int s = 0; s < S; ++s) issue();

    int done = 0, ds = 0;                 // tiles of this warp already computed, the stage of the next
    uint32_t parity = 0;
    int own_abort = 0;
    int first = cum[b].x * per, each = cum[b + 1].x - cum[b].x;   // of the request: first tile, tiles per unit
#pragma unroll 1
    for (;;) {
        const int us = first + unit * each, ue = us + each;
        const int head = P.row_tiles == 1 ? unit : unit / P.row_tiles, rt = unit - head * P.row_tiles;
        const int rows = min(R, P.rows - rt * R);                    // live rows of this unit
        const int row0 = b * P.rows + rt * R;
        const int len = len_of(b);

        QFrag<BITS, D, NT> Q;
        load_q<BITS, D, NT, T>(P, Q, row0, rows, head, n, t);
        State<D, NT> A;
        int seen[NT][2];   // tokens that rows 2 t, 2 t + 1 see
        A.ks = kUnset | kNoScales;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) A.oz[nt][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                A.m[nt][i] = -INFINITY;
                A.l[nt][i] = A.ref[nt][i] = 0.f;
                const int r = rt * R + 8 * nt + 2 * t + i;
                seen[nt][i] = P.prefix == 1 ? len : len - P.tokens + 1 + min(r / P.group, P.tokens - 1);
            }
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) A.o[nt][k][i] = 0.f;
        }
        const int whole = (P.prefix == 1 ? len : len - P.tokens + 1) - kKvTile;   // later tiles: not every row sees all
        const int2 gap = gap_of(len);
        const int lowest = len - P.tokens - P.window + 1;   // (kWin) the first row's window begins here

        const int upto = min(ue, g1) - g0 - warp;   // tiles of this warp: W * done < upto
        int j0 = (g0 + warp + W * done - us) * kKvTile;
#pragma unroll 1
        for (; W * done < upto; ++done, j0 += W * kKvTile) {
            mbar_wait_bounded(bars + 8 * ds, parity, &own_abort, P.status);
            if (there >> ds & 1u) {
                const uint8_t* tile = smem + (warp * S + ds) * L::kBytes;
                constexpr bool kFine = IsHalf<T>::value;
                const int at = kWin && j0 >= gap.x * kKvTile ? j0 + gap.y * kKvTile : j0;
                if (at > whole || (kWin && at < len - P.window && at + kKvTile > P.sinks))
                    tile_step<BITS, D, NT, true, kFine, kWin>(tile, Q, A, at, len, seen, lane, P.window, P.sinks, lowest);
                else tile_step<BITS, D, NT, false, kFine, kWin>(tile, Q, A, at, len, seen, lane, 0, 0, 0);
            }
            __syncwarp();   // all lanes have read the stage: it may be filled again
            issue();
            if (++ds == S) ds = 0, parity ^= 1u;
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
                for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * R + r].x);
                const float ref = top == -INFINITY ? 0.f : top;
                for (int w = 0; w < W; ++w) l += ml[w * R + r].y * ex2(ml[w * R + r].x - ref);
                fac[nt][i] = ex2(A.m[nt][i] - ref);
                if (warp == 0 && n == 0) total_ml[r] = make_float2(top, l);
            }
        auto put = [&](bool add) {   // this warp's rows into (or onto) slot warp % (W / 2)
            float* dst = red + (warp % (W / 2)) * R * M::kPitch;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                    const float up = pow2i(24 - ks_of(A.ks, k >> 1));
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
        if (warp >= W / 2) put(false);
        __syncthreads();
        if (warp < W / 2) put(true);
        __syncthreads();

        const bool all_here = us >= g0 && ue <= g1;
        float* slot = P.part + (2 * c + (us >= g0 ? 1 : 0)) * (int64_t)(R * (D + 2));
        constexpr int V = D / 32;   // a warp per row
        for (int r = warp; r < rows; r += W) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float* a = red + r * M::kPitch + V * lane + i;
                v[i] = a[0] + a[R * M::kPitch];
                if (W == 8) v[i] += a[2 * R * M::kPitch] + a[3 * R * M::kPitch];
            }
            if (all_here) {
                finish_row<D, T>(P, row0 + r, head, total_ml[r].x, total_ml[r].y, v, lane);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) slot[r * D + V * lane + i] = v[i];
            }
        }
        if (!all_here) {
            if (tid < rows) *reinterpret_cast<float2*>(slot + R * D + 2 * tid) = total_ml[tid];
            // the blocks that share the unit
            const int from = costly(b) * per + unit * (each + kCost) + kCost;
            const int c0 = pieces ? c - piece : shares.of(from), c1 = pieces ? c0 + of - 1 : shares.of(from + each - 1);
            unsigned* count = P.counters + (int64_t)b * per + unit;
            __syncthreads();
            // (release of what the block wrote before the barrier, acquire of what the others did)
            if (tid == 0) s_last = arrive_gpu(count) == (unsigned)(c1 - c0);
            __syncthreads();
            if (s_last) {
                join<D, R, W, T>(P, c0, c1, warp, lane, rows, row0, head);
                if (tid == 0) *count = 0;
            }
        }
        if (ue >= g1) break;
        if (++unit == per) {
            unit = 0;
            ++b;
            first = cum[b].x * per;
            each = cum[b + 1].x - cum[b].x;
        }
        __syncthreads();   // the sums' buffers are free again
    }
}

// Requests that the shared memory of a launch has room for: a few sizes, so that few are ever asked about.
int cum_room(int requests) { return requests <= 64 ? 64 : requests <= 256 ? 256 : kMaxAttnBatch; }

// Blocks of a kernel that fit on the device at once (0 on error); sets its shared-memory attribute,
// which only rises.  Kept per kernel, device and size.
template <int BITS, int D, int NT, int W, class T, bool kWin>
int attn_blocks(int device, int num_sms, int requests) {
    static std::mutex mu;
    static int known[kMaxDevices][3] = {}, most[kMaxDevices] = {};
    if (device < 0 || device >= kMaxDevices) return 0;
    const int room = cum_room(requests), smem = AttnSmem<BITS, D, NT, W>::kCum + 8 * (room + 1);
    const std::lock_guard<std::mutex> lock(mu);
    int& blocks = known[device][room == 64 ? 0 : room == 256 ? 1 : 2];
    if (blocks == 0) {
        if (smem > most[device]) {
            if (cudaFuncSetAttribute(attn_kernel<BITS, D, NT, W, T, kWin>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return 0;
            most[device] = smem;
        }
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kernel<BITS, D, NT, W, T, kWin>, 32 * W, smem) != cudaSuccess) return 0;
        blocks = n * num_sms;
    }
    return blocks;
}

template <int BITS, int D, int NT, int W, class T, bool kWin>
lq_status run(lq_handle h, AttnParams& P, Scratch& s) {
    constexpr int R = 8 * NT;
    P.row_tiles = (P.rows + R - 1) / R;
    const int blocks = attn_blocks<BITS, D, NT, W, T, kWin>(h->device, h->num_sms, P.requests);
    if (blocks < 1) return LQ_ERR_CUDA;
    // (tile indices are 32-bit, quotients of units below 2^20)
    if (((int64_t)P.max_len / kKvTile + 2 + kUnitCost<W>) * P.requests * P.cache.kv_heads * P.row_tiles > 0x7fffffffLL) return LQ_ERR_UNSUPPORTED;
    if (blocks > 1024 || (int64_t)P.cache.kv_heads * P.row_tiles >= (1 << 20)) return LQ_ERR_UNSUPPORTED;
    if ((size_t)P.requests * P.cache.kv_heads * P.row_tiles > h->num_counters) return LQ_ERR_WORKSPACE;
    s.need = (size_t)blocks * 2 * R * (D + 2) * sizeof(float);
    if (s.need > s.room) return LQ_ERR_WORKSPACE;
    if (!s.launch) return LQ_OK;
    P.part = reinterpret_cast<float*>(s.at);
    return launch_overlapped(attn_kernel<BITS, D, NT, W, T, kWin>, blocks, 32 * W,
                             AttnSmem<BITS, D, NT, W>::kCum + 8 * (cum_room(P.requests) + 1), s.stream, P);
}

template <int BITS, int D, int NT, bool kWin>
lq_status run_typed(lq_handle h, AttnParams& P, bool bf16, Scratch& s) {
    const int64_t units = (int64_t)P.requests * P.cache.kv_heads * ((P.rows + 8 * NT - 1) / (8 * NT));
    if (units > 2 * h->num_sms)
        return bf16 ? run<BITS, D, NT, 4, __nv_bfloat16, kWin>(h, P, s) : run<BITS, D, NT, 4, __half, kWin>(h, P, s);
    return bf16 ? run<BITS, D, NT, 8, __nv_bfloat16, kWin>(h, P, s) : run<BITS, D, NT, 8, __half, kWin>(h, P, s);
}

template <int BITS, int D, bool kWin>
lq_status run_rows(lq_handle h, AttnParams& P, bool bf16, Scratch& s) {
    // one n = 8 tile of rows where 8 hold them, two otherwise (a second tile costs a third more issue slots per key)
    return P.rows <= 8 ? run_typed<BITS, D, 1, kWin>(h, P, bf16, s) : run_typed<BITS, D, 2, kWin>(h, P, bf16, s);
}

template <bool kWin>
lq_status run_shape(lq_handle h, AttnParams& P, int bits, int D, bool bf16, Scratch s) {
    if (D == 128) return bits == 4 ? run_rows<4, 128, kWin>(h, P, bf16, s) : run_rows<8, 128, kWin>(h, P, bf16, s);
    return bits == 4 ? run_rows<4, 64, kWin>(h, P, bf16, s) : run_rows<8, 64, kWin>(h, P, bf16, s);
}

}  // namespace
}  // namespace lq
