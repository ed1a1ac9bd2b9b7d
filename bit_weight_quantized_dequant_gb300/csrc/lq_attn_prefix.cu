// Attention of many query rows over one shared prefix, on the tensor-memory tensor cores.
//
// A prefix that all requests of a batch share meets all their rows: batch * tokens * group rows
// per kv head, hundreds of them, so the work is a dense contraction and no longer the cache's
// bytes.  A block takes 128 rows of one kv head and a range of keys, 64 at a time:
//   S [128 rows][64 keys] = Q K^T      Q in tensor memory, K in shared memory
//   P = 2^(S f - m)                    a thread per row, S read from and P written to tensor memory
//   O [128 rows][D]      += P V        P in tensor memory, V [D][64 keys] in shared memory
// by one-CTA tcgen05.mma (M 128, N 64 and N D, binary16 operands, fp32 sums).
//
// Scores keep fp32 precision.  K's code part S c is the sum of two binary16 values, its rounding
// and what that left out (one fused multiply-add gives it exactly), each multiplied; its offset
// part is one more MMA of 16 columns, Z by the group sums of q in two binary16 terms.  K is held
// times 2^-2 and V times 2^-1, so that nothing within the cache's range overflows; V is rounded
// to binary16 (absolute error 2^-24 below 2^-13).
//
// Roles (18 warps): one loads tiles by bulk copies; one thread issues the MMAs; eight expand
// codes (four K, four V: a 16-token tile each); eight do the softmax, as two groups of 128 threads
// that take the key blocks in turn, each with its own S/P buffer, running maximum and O (two O
// accumulators need no exchange between the groups until the unit's end).  All MMAs come from one
// thread and run in its order, so one barrier per buffer and direction suffices: S full (which
// also frees K's stage and, being later in order, says that P's buffer was read), P full, O done
// (which frees V's stage).  Every wait is bounded; a role whose wait ran out goes on with what is
// there, so every loop and barrier still ends, and the status word reports it.

#include <algorithm>
#include <mutex>
#include <vector>

#include "lq_attn.cuh"
#include "lq_tcgen05.cuh"

namespace lq {
namespace {

constexpr int kRows = 128;          // rows of a unit
constexpr int kKeys = 64;           // keys of a block
constexpr int kTiles = kKeys / kKvTile;
constexpr int kRaw = 3;             // key blocks of cache bytes in flight
constexpr int kSoftWarps = 8, kDqWarps = 8;
constexpr int kSoft0 = 0, kDq0 = kSoft0 + kSoftWarps, kMmaWarp = kDq0 + kDqWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + 1);
// tensor memory columns
constexpr int kTmemCols = 512;
constexpr int kColS = 0;            // 2 x 64: S, then P in the first 32 of each
constexpr int kColO = 128;          // 2 x D
constexpr int kColQ = 384;          // D / 2
constexpr int kColZ = 448;          // 8 (group sums of q), 32 written
static_assert(kColO + 2 * 128 <= kColQ && kColQ + 64 <= kColZ && kColZ + 32 <= kTmemCols, "tensor memory");

template <int BITS, int D>
struct PreSmem {
    using L = KvLayout<BITS, D>;
    static constexpr int kAtoms = D / 64;                        // 128-byte rows of 64 dimensions
    static constexpr int kAtom = kKeys * 128;                    // one of them for all keys of a block
    static constexpr int kKStage = (2 * kAtoms + 1) * kAtom;     // K rounded, K's rest, Z
    static constexpr int kVStage = D * 128;                      // [D][64 keys]
    static constexpr int kRawStage = (kTiles * L::kBytes + 127) / 128 * 128;
    static constexpr int kK = 0;
    static constexpr int kV = kK + 2 * kKStage;
    static constexpr int kRawOff = kV + 2 * kVStage;
    static constexpr int kMl = kRawOff + kRaw * kRawStage;       // [2 groups][rows] m, l
    static constexpr int kF = kMl + 2 * kRows * 8;               // [rows] score factors
    static constexpr int kBars = kF + kRows * 4;
    static constexpr int kNumBars = 2 * kRaw + 2 * 5 + 1;
    static constexpr int kSize = 1024 + kBars + 8 * kNumBars;
    static_assert(kSize <= 227 * 1024 && kBars % 8 == 0, "shared memory");
};

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }   // the softmax warps
__device__ __forceinline__ void sts128(uint8_t* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

// Whole numbers (binary16 pairs) of a word's codes: 4-bit r = 0..3: nibbles (r, r + 4); 8-bit
// r = 0, 1: bytes (r, r + 2).
template <int BITS>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int r) {
    if (BITS == 4) {
        const uint32_t y = r & 2 ? w >> 8 : w;
        if (r & 1) return hadd2((y & 0x00f000f0u) | 0x54005400u, 0xd400d400u);   // 64 + c, less 64
        return hadd2((y & 0x000f000fu) | 0x64006400u, 0xe400e400u);              // 1024 + c, less 1024
    }
    return hadd2(prmt(w, 0x64646464u, r ? 0x4341 : 0x4240), 0xe400e400u);
}

// Keys of one tile: [token][dims] rows of the K stage, in the order of the words' pairs (Q's columns
// follow it).  left: tokens of the prefix from the tile's first on.
template <int BITS, int D>
__device__ __forceinline__ void expand_keys(const uint8_t* tile, uint8_t* stage, int tile_no, int left, int lane) {
    using L = KvLayout<BITS, D>;
    using M = PreSmem<BITS, D>;
    constexpr int G = D / 32, WK = L::WK, U = WK / G;   // U words of a group (1 or 2)
    const int n = lane >> 2, t = lane & 3;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int tok = n + 8 * hf, row = 16 * tile_no + tok;   // row & 7 == n
        alignas(16) uint32_t kw[WK];
        if (WK >= 4) {
#pragma unroll
            for (int q = 0; q < WK; q += 4)
                *reinterpret_cast<uint4*>(kw + (q & (WK - 1))) = lds128(tile + kv_word_at(lane, hf * WK + q));
        } else {
            *reinterpret_cast<uint2*>(kw) = lds64(tile + kv_word_at(lane, hf * WK));
        }
        const uint32_t keep = tok < left ? 0xffffffffu : 0u;     // past the end: zeros, whatever lies there
        uint32_t s[G / 2], z[G / 2];
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
            s[i] = hmul2(lds32(tile + L::kKs + tok * G * 2 + 4 * i) & keep, 0x34003400u);   // 2^-2
            z[i] = hmul2(lds32(tile + L::kKz + tok * G * 2 + 4 * i) & keep, 0x34003400u);
        }
        uint8_t* base = stage + row * 128;
#pragma unroll
        for (int st = 0; st < G; ++st) {
            // odd tokens take their groups in the other order, so that eight lanes write to eight places
            const int g = st ^ (n & 1);
            const uint32_t pair = s[st >> 1], s2 = prmt(pair, 0, g & 1 ? 0x3232 : 0x1010);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t w0 = kw[U * st + u], w1 = kw[U * (st ^ 1) + u], w = n & 1 ? w1 : w0;
#pragma unroll
                for (int r = 0; r < 4 / U; ++r) {
                    const uint32_t c = code_pair<BITS>(w, r);
                    const uint32_t p = hmul2(c, s2);
                    hi[u * (4 / U) + r] = p;
                    lo[u * (4 / U) + r] = hfma2(c, s2, p ^ 0x80008000u);   // c S - p, exactly
                }
            }
            const int ch = 4 * g + t;
            uint8_t* at = base + (ch >> 3) * M::kAtom + (((ch & 7) ^ n) << 4);
            sts128(at, hi[0], hi[1], hi[2], hi[3]);
            sts128(at + M::kAtoms * M::kAtom, lo[0], lo[1], lo[2], lo[3]);
        }
        if (t == 0) {   // Z against both terms of the group sums
            uint8_t* at = base + 2 * M::kAtoms * M::kAtom + (n << 4);
            if (G == 4) sts128(at, z[0], z[G / 2 - 1], z[0], z[G / 2 - 1]);
            else sts128(at, z[0], z[0], 0u, 0u);
        }
    }
}

// Values of one tile: [dimension][keys] rows of the V stage, two keys per word.
template <int BITS, int D>
__device__ __forceinline__ void expand_values(const uint8_t* tile, uint8_t* stage, int tile_no, int left, int lane) {
    using L = KvLayout<BITS, D>;
    constexpr int G = D / 32, WV = L::WV;
    const int n = lane >> 2, t = lane & 3;
    alignas(16) uint32_t vw[4 * WV];
#pragma unroll
    for (int c = 0; c < L::kChunks; ++c)
        *reinterpret_cast<uint4*>(vw + 4 * c) = lds128(tile + L::kVc + 512 * c + 16 * lane);
    const uint32_t keep[2] = {(2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u),
                              (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u)};
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint2 sv = lds64(tile + L::kVs + g * 32 + 8 * t), zv = lds64(tile + L::kVz + g * 32 + 8 * t);
        const uint32_t s[2] = {hmul2(sv.x & keep[0], 0x38003800u), hmul2(sv.y & keep[1], 0x38003800u)};   // 2^-1
        const uint32_t z[2] = {hmul2(zv.x & keep[0], 0x38003800u), hmul2(zv.y & keep[1], 0x38003800u)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int slab = 4 * g + k, wi = slab % WV, e = slab / WV, d = 8 * slab + n;   // (d & 7 == n)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t wa = vw[2 * half * WV + wi], wb = vw[(2 * half + 1) * WV + wi];
                uint32_t c;
                if (BITS == 4) {
                    const uint32_t y = prmt(wa, wb, e < 4 ? 0x5410 : 0x7632), w = (e & 2) ? y >> 8 : y;
                    c = (e & 1) ? hadd2((w & 0x00f000f0u) | 0x54005400u, 0xd400d400u)
                                : hadd2((w & 0x000f000fu) | 0x64006400u, 0xe400e400u);
                } else {
                    const uint32_t y = prmt(wa, wb, e < 2 ? 0x5410 : 0x7632), w = (e & 1) ? y >> 8 : y;
                    c = hadd2((w & 0x00ff00ffu) | 0x64006400u, 0xe400e400u);
                }
                *reinterpret_cast<uint32_t*>(stage + d * 128 + (((2 * tile_no + half) ^ n) << 4) + 4 * t) = hfma2(c, s[half], z[half]);
            }
        }
    }
}

// One key block's scores of a row: maximum, reference, P.
struct RowSum {
    float m, l, ref;
};

template <int BITS, int D, class T>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ AttnParams P) {
    using L = KvLayout<BITS, D>;
    using M = PreSmem<BITS, D>;
    constexpr int G = D / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // (the swizzle's 1024-byte atoms)
    float2* ml = reinterpret_cast<float2*>(base + M::kMl);
    float* factors = reinterpret_cast<float*>(base + M::kF);
    __shared__ uint32_t s_tmem;
    __shared__ int s_last;
    __shared__ volatile uint32_t s_there[8];   // a block's tiles that are in the cache (no role is 8 blocks ahead of another)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const uint32_t bars = smem_u32(base + M::kBars);
    const uint32_t raw_full = bars, raw_empty = raw_full + 8 * kRaw, k_full = raw_empty + 8 * kRaw, v_full = k_full + 16;
    const uint32_t s_full = v_full + 16, p_full = s_full + 16, o_done = p_full + 16, q_full = o_done + 16;
    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, kDqWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full + 8 * b, kTiles);
            mbar_init(v_full + 8 * b, kTiles);
            mbar_init(s_full + 8 * b, 1);
            mbar_init(p_full + 8 * b, 4);
            mbar_init(o_done + 8 * b, 1);
        }
        mbar_init(q_full, 4);
        fence_mbar_init();
    }
    // the Z rows' second 16 bytes multiply nothing: zero for good
    for (int i = tid; i < 2 * kKeys; i += kThreads)
        sts128(base + M::kK + (i / kKeys) * M::kKStage + 2 * M::kAtoms * M::kAtom + (i % kKeys) * 128 + ((1 ^ (i & 7)) << 4), 0, 0, 0, 0);
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    pdl_wait();

    // this block's key blocks of the sequence of all (kv head, row tile) units' blocks
    const int each = (P.max_len + kKeys - 1) / kKeys;
    const int total = each * P.cache.kv_heads * P.row_tiles, C = gridDim.x, c = blockIdx.x;
    const int q = total / C, rem = total - q * C;
    const int g0 = q * c + min(c, rem), g1 = q * (c + 1) + min(c + 1, rem), blocks = g1 - g0;
    int own_abort = 0;
    auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait_bounded(bar, parity & 1u, &own_abort, P.status); };

    if (warp == kLoadWarp) {
        // ---------------------------------------------------------------- tiles into the raw ring
        const uint8_t* src = nullptr;
        for (int i = 0; i < blocks; ++i) {
            if (i % 8 == 0) {   // addresses of eight blocks' tiles, one per lane
                const int gb = g0 + i + lane / kTiles;
                src = nullptr;
                if (gb < g1) {
                    const int unit = gb / each, tile = (gb - unit * each) * kTiles + lane % kTiles, head = unit / P.row_tiles;
                    if (tile * kKvTile < P.max_len) {
                        const int pi = tile / P.cache.tiles_per_page, page = __ldg(P.block_table + pi);
                        if (page < 0 || page >= P.cache.num_pages) atomicOr(P.status, kStatusIndex);
                        else
                            src = P.cache.pages + (((int64_t)page * P.cache.kv_heads + head) * P.cache.tiles_per_page +
                                                   (tile - pi * P.cache.tiles_per_page)) * (int64_t)L::kBytes;
                    }
                }
            }
            const int s = i % kRaw;
            if (i >= kRaw) wait(raw_empty + 8 * s, i / kRaw - 1);
            __syncwarp();
            const uint32_t there = (__ballot_sync(0xffffffffu, src != nullptr) >> (i % 8 * kTiles)) & ((1u << kTiles) - 1u);
            if (lane == 0) {
                s_there[i & 7] = there;
                if (there) mbar_arrive_expect_tx(raw_full + 8 * s, __popc(there) * L::kBytes);
                else mbar_arrive(raw_full + 8 * s);
            }
            __syncwarp();
            if (lane / kTiles == i % 8 && src)
                bulk_load(smem_u32(base + M::kRawOff + s * M::kRawStage) + lane % kTiles * L::kBytes, src, L::kBytes, raw_full + 8 * s);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- all MMAs, one thread
        if (lane == 0) {
            const uint32_t idS = idesc_f16(false, kRows, kKeys), idO = idesc_f16(false, kRows, D);
            const uint32_t ks = smem_u32(base + M::kK), vs = smem_u32(base + M::kV);
            auto scores = [&](int i) {
                const int b = i & 1;
                const uint32_t d = tmem + kColS + kKeys * b, k = ks + b * M::kKStage;
                wait(k_full + 8 * b, i >> 1);
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int st = 0; st < D / 16; ++st)
                        tc_mma_f16_ts(d, tmem + kColQ + 8 * st,
                                      smem_desc_sw128(k + (part * M::kAtoms + st / 4) * M::kAtom + 32 * (st % 4)), idS, (part | st) != 0);
                tc_mma_f16_ts(d, tmem + kColZ, smem_desc_sw128(k + 2 * M::kAtoms * M::kAtom), idS, 1);
                tc_commit(s_full + 8 * b);
            };
            int done = 0;   // blocks of earlier units
            for (int u = 0; done < blocks; ++u) {
                const int unit = (g0 + done) / each, nb = min((unit + 1) * each, g1) - (g0 + done);
                wait(q_full, u);
                tc_fence_after();
                scores(done);
                if (nb > 1) scores(done + 1);
                for (int j = 0; j < nb; ++j) {
                    const int i = done + j, b = i & 1;
                    wait(v_full + 8 * b, i >> 1);
                    wait(p_full + 8 * b, i >> 1);
                    tc_fence_after();
#pragma unroll
                    for (int st = 0; st < kKeys / 16; ++st)
                        tc_mma_f16_ts(tmem + kColO + D * b, tmem + kColS + kKeys * b + 8 * st,
                                      smem_desc_sw128(vs + b * M::kVStage + 32 * st), idO, j >= 2 || st != 0);
                    tc_commit(o_done + 8 * b);
                    if (j + 2 < nb) scores(i + 2);
                }
                done += nb;
            }
        }
        __syncwarp();
    } else if (warp >= kDq0) {
        // ---------------------------------------------------------------- codes to operands
        const int w = warp - kDq0, tile_no = w % kTiles;
        const bool keys = w < kTiles;
        for (int i = 0; i < blocks; ++i) {
            const int s = i % kRaw, b = i & 1, gb = g0 + i, kb = gb - gb / each * each;
            wait(raw_full + 8 * s, i / kRaw);
            if (i >= 2) wait((keys ? s_full : o_done) + 8 * b, (i >> 1) - 1);   // the stage's last MMAs have read it
            const uint8_t* tile = base + M::kRawOff + s * M::kRawStage + tile_no * L::kBytes;
            const int left = s_there[i & 7] >> tile_no & 1u ? P.max_len - kb * kKeys - tile_no * kKvTile : 0;
            if (keys) expand_keys<BITS, D>(tile, base + M::kK + b * M::kKStage, tile_no, left, lane);
            else expand_values<BITS, D>(tile, base + M::kV + b * M::kVStage, tile_no, left, lane);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive((keys ? k_full : v_full) + 8 * b);
                mbar_arrive(raw_empty + 8 * s);
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax: a thread per row
        const int grp = warp >> 2, r = 32 * (warp & 3) + lane;         // group of the blocks with i & 1 == grp
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        int done = 0;
        for (int u = 0; done < blocks; ++u) {
            const int unit = (g0 + done) / each, us = unit * each, ue = us + each, nb = min(ue, g1) - (g0 + done);
            const int head = unit / P.row_tiles, rt = unit - head * P.row_tiles, rows = min(kRows, P.all_rows - rt * kRows);
            if (grp == 0) {
                // Q, scaled by a power of two into [2^9, 2^10), its columns in the order of K's rows
                float top = 0.f;
                const int row = rt * kRows + r, bt = row / P.group;
                const uint16_t* src = static_cast<const uint16_t*>(P.q) + bt * P.q_stride + (int64_t)(head * P.group + (row - bt * P.group)) * D;
                const bool live = r < rows;
#pragma unroll 4
                for (int k = 0; k < D / 8; ++k) {
                    const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(elem_to_float<T>((uint16_t)(w[e >> 1] >> (16 * (e & 1))))));
                }
                int e = top > 0.f ? 9 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
                e = min(max(e, -120), 120);
                const float up = pow2i(e);
                factors[r] = P.scale_log2 * pow2i(-e) * 4.f;           // (K is held times 2^-2)
                uint32_t z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {                     // 64 dimensions: 32 columns
                    uint32_t o[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 64 * h + 8 * k) : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = elem_to_float<T>((uint16_t)(w[i >> 1] >> (16 * (i & 1)))) * up;
                        if (BITS == 4) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[4 * k + i] = pack_half2_rn(f[i], f[i + 4]);
                        } else {
                            o[4 * k] = pack_half2_rn(f[0], f[2]), o[4 * k + 1] = pack_half2_rn(f[1], f[3]);
                            o[4 * k + 2] = pack_half2_rn(f[4], f[6]), o[4 * k + 3] = pack_half2_rn(f[5], f[7]);
                        }
                    }
                    tmem_st32(lanes + kColQ + 32 * h, o);
#pragma unroll
                    for (int gg = 0; gg < 2; ++gg) {                   // sums of the rounded values of a group
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 p = unpack2(o[16 * gg + i]);
                            sum += p.x + p.y;
                        }
                        const int g = 2 * h + gg;
                        const __half hi = __float2half_rn(sum), lo = __float2half_rn(sum - __half2float(hi));
                        z[g >> 1] |= (uint32_t)__half_as_ushort(hi) << (16 * (g & 1));
                        z[G / 2 + (g >> 1)] |= (uint32_t)__half_as_ushort(lo) << (16 * (g & 1));
                    }
                }
                tmem_st32(lanes + kColZ, z);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            soft_sync();   // the factors
            const float f = factors[r];
            RowSum A{-INFINITY, 0.f, 0.f};
            for (int j = (done & 1) == grp ? 0 : 1; j < nb; j += 2) {
                const int i = done + j;
                wait(s_full + 8 * grp, i >> 1);
                tc_fence_after();
                const uint32_t col = lanes + kColS + kKeys * grp;
                float x[kKeys];
                tmem_ld32(col, reinterpret_cast<uint32_t(&)[32]>(x[0]));
                tmem_ld32(col + 32, reinterpret_cast<uint32_t(&)[32]>(x[32]));
                const int left = P.max_len - (g0 + i - us) * kKeys;    // keys of the prefix from the block's first on
                const uint32_t there = s_there[i & 7];
                if (left < kKeys || there != (1u << kTiles) - 1u) {
#pragma unroll
                    for (int k = 0; k < kKeys; ++k)
                        if (k >= left || !(there >> (k / kKvTile) & 1u)) x[k] = -INFINITY;
                }
                float mx = x[0];
#pragma unroll
                for (int k = 1; k < kKeys; ++k) mx = fmaxf(mx, x[k]);
                mx *= f;
                const bool move = mx > A.m + kTau;
                if (__any_sync(0xffffffffu, move)) {
                    const float now = move ? mx : A.m, a = A.m == now ? 1.f : ex2(A.m - now);
                    if (j >= 2 && __any_sync(0xffffffffu, A.m != now)) {
                        // O's last addition was earlier in the MMA thread's order than S, so it is complete
#pragma unroll 1
                        for (int d = 0; d < D; d += 32) {
                            uint32_t o[32];
                            tmem_ld32(lanes + kColO + D * grp + d, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                            tmem_st32(lanes + kColO + D * grp + d, o);
                        }
                    }
                    A.l *= a;
                    A.m = now;
                    A.ref = now == -INFINITY ? 0.f : now - kPBits;
                }
                uint32_t p[kKeys / 2];
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int k = 0; k < kKeys; k += 2) {
                    const float a = ex2(fmaf(x[k], f, -A.ref)), b = ex2(fmaf(x[k + 1], f, -A.ref));
                    l0 += a;
                    l1 += b;
                    p[k / 2] = pack_half2_rn(a, b);
                }
                A.l += l0 + l1;
                tmem_st32(col, p);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * grp);
            }

            // ---- the two groups' sums of the unit: each thread half of its row's dimensions ----
            ml[grp * kRows + r] = make_float2(A.m, A.l);
            soft_sync();
            const int i1 = done + nb - 1;                              // the unit's last block
            wait(o_done + 8 * (i1 & 1), i1 >> 1);
            if (nb > 1) wait(o_done + 8 * ((i1 - 1) & 1), (i1 - 1) >> 1);
            tc_fence_after();
            const float2 e0 = ml[r], e1 = ml[kRows + r];
            const float top = fmaxf(e0.x, e1.x), ref = top == -INFINITY ? 0.f : top;
            const float f0 = ex2(e0.x - ref), f1 = ex2(e1.x - ref), l = e0.y * f0 + e1.y * f1;
            const bool has0 = nb > 1 || (done & 1) == 0, has1 = nb > 1 || (done & 1) == 1;
            const bool all_here = us >= g0 && ue <= g1;
            float* slot = P.part + (2 * c + (us >= g0 ? 1 : 0)) * (int64_t)(kRows * (D + 2));
            const RowOut<D, T> out(P, rt * kRows + min(r, rows - 1), head, top, l, all_here && grp == 0 && r < rows);
#pragma unroll 1
            for (int d = grp * (D / 2); d < (grp + 1) * (D / 2); d += 32) {
                uint32_t a[32], b[32];
                tmem_ld32(lanes + kColO + d, a);
                tmem_ld32(lanes + kColO + D + d, b);
                if (r < rows) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)                    // (V is held times 2^-1)
                            v[i] = 2.f * ((has0 ? __uint_as_float(a[k + i]) * f0 : 0.f) + (has1 ? __uint_as_float(b[k + i]) * f1 : 0.f));
                        if (all_here) out.store(P, d + k, v);
                        else *reinterpret_cast<float4*>(slot + r * D + d + k) = make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            if (!all_here) {
                if (grp == 0 && r < rows) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(top, l);
                auto block_of = [&](int at) { return at < rem * (q + 1) ? at / (q + 1) : rem + (at - rem * (q + 1)) / q; };
                const int c0 = block_of(us), c1 = block_of(ue - 1);
                __threadfence();
                soft_sync();
                if (tid == 0) s_last = atomicAdd(P.counters + unit, 1u) == (unsigned)(c1 - c0);
                soft_sync();
                if (s_last) {
                    __threadfence();
                    join<D, kRows, kSoftWarps, T>(P, c0, c1, warp, lane, rows, rt * kRows, head);
                    if (tid == 0) P.counters[unit] = 0;
                }
            }
            tc_fence_before();
            soft_sync();   // both groups are done with O, the factors and the sums
            done += nb;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int BITS, int D, class T>
lq_status run(lq_handle h, AttnParams& P, char* scratch, size_t room, cudaStream_t stream) {
    using M = PreSmem<BITS, D>;
    static std::mutex mu;
    static std::vector<int> ready;   // per device: the shared-memory attribute is set
    {
        std::lock_guard<std::mutex> lock(mu);
        if ((int)ready.size() <= h->device) ready.resize(h->device + 1, 0);
        if (!ready[h->device]) {
            if (M::kSize > h->max_smem_optin ||
                cudaFuncSetAttribute(prefix_kernel<BITS, D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kSize) != cudaSuccess)
                return LQ_ERR_CUDA;
            ready[h->device] = 1;
        }
    }
    P.row_tiles = (P.all_rows + kRows - 1) / kRows;
    const int64_t units = (int64_t)P.cache.kv_heads * P.row_tiles, total = units * ((P.max_len + kKeys - 1) / kKeys);
    if (total > 0x7fffffffLL) return LQ_ERR_UNSUPPORTED;
    const int blocks = (int)std::min<int64_t>(h->num_sms, total);
    if ((size_t)units > h->num_counters || (size_t)blocks * 2 * kRows * (D + 2) * sizeof(float) > room) return LQ_ERR_WORKSPACE;
    P.part = reinterpret_cast<float*>(scratch);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = M::kSize;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefix_kernel<BITS, D, T>, P) == cudaSuccess ? LQ_OK : LQ_ERR_CUDA;
}

}  // namespace

bool prefix_tc_takes(int rows, int prefix_len) { return rows >= 64 && prefix_len >= 256; }

lq_status launch_prefix_tc(lq_handle h, AttnParams& P, int bits, int D, bool bf16, char* scratch, size_t room, cudaStream_t stream) {
    if (D == 128) {
        if (bits == 4) return bf16 ? run<4, 128, __nv_bfloat16>(h, P, scratch, room, stream) : run<4, 128, __half>(h, P, scratch, room, stream);
        return bf16 ? run<8, 128, __nv_bfloat16>(h, P, scratch, room, stream) : run<8, 128, __half>(h, P, scratch, room, stream);
    }
    if (bits == 4) return bf16 ? run<4, 64, __nv_bfloat16>(h, P, scratch, room, stream) : run<4, 64, __half>(h, P, scratch, room, stream);
    return bf16 ? run<8, 64, __nv_bfloat16>(h, P, scratch, room, stream) : run<8, 64, __half>(h, P, scratch, room, stream);
}

}  // namespace lq
