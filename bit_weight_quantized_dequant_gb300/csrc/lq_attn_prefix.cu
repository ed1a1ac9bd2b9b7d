// Attention of many query rows over one shared prefix, on the tensor-memory tensor cores.
//
// A prefix that all requests of a batch share meets all their rows: batch * tokens * group rows
// per kv head, hundreds of them, so the work is a dense contraction and no longer the cache's
// bytes.  A block takes 128 rows of one kv head and a range of keys, 128 at a time:
//   S [128 rows][128 keys] = Q K^T     Q in tensor memory, K in shared memory
//   P = 2^(S f - m)                    S read from and P written to tensor memory
//   O [128 rows][D]       += P V       P in tensor memory, V [D][128 keys] in shared memory
// by one-CTA tcgen05.mma (M 128, N 128 and N D, binary16 operands, fp32 sums).  An M = 128 MMA
// takes 62 cycles at N = 64 and 64 at N = 128 (measured), so narrower key blocks waste the pipe.
//
// Scores keep fp32 precision.  K's code part S c is the sum of two binary16 values, its rounding
// and what that left out (one fused multiply-add gives it exactly), each multiplied; its offset
// part is one more MMA of 16 columns, Z by the group sums of q in two binary16 terms.  V is rounded
// to binary16 (absolute error 2^-25 below 2^-14).  A group that spans all of binary16's range (clamped
// infinities) has terms past its end.  They are clamped, two instructions per pair of keys' terms and
// one per pair of values (3 us of 107); a branch around them cost 5, and scaling S down instead
// costs it bits where it is small.
//
// Roles (27 warps of 28): two load keys' and values' bytes by bulk copies, each into a ring of its own
// (values wait for the O before them, keys run two blocks ahead); one issues the MMAs; sixteen expand codes (eight K,
// eight V, a 16-token tile each); eight do the softmax, two threads per row with half of the keys each,
// which share the row's reference (one barrier of their two warps per key block tells whether it has
// to move).  K and S have two stages, so that the next block's scores are computed while this one's
// softmax runs; V has one: its next block is expanded while those scores are.  All MMAs come from one
// thread and run in its order, so few barriers suffice: S full (which also frees K's stage and, being
// later in order, says that P's buffer was read), P full, O done (which frees V's stage).  A wait tells a
// barrier's phases apart by their parity alone, so each role waits for every phase of a barrier in turn, and
// arrives on what the next one needs only after that.  Every wait is bounded; a role whose wait ran out goes
// on with what is there, so every loop and barrier still ends, and the status word reports it.
//
// Measured with 48 requests of 64 query heads over 8 (128 dimensions, bf16) and 32100 shared tokens in 4
// bits: 85 us, and 116 the whole call (338 with the kernel of lq_attn.cu for the prefix).  A block of 128 keys takes
// 3870 cycles, of which its MMAs are 1607 (tensor pipe 41 %): codes becoming operands, which each of the three row
// tiles of a kv head expands for itself, and the softmax bound it (issue 65 %, ALU 56 %).

#include <algorithm>
#include <mutex>

#include "lq_attn_tc.cuh"

namespace lq {
namespace {

constexpr int kRows = 128;          // rows of a unit
constexpr int kKeys = kTcKeys;      // keys of a block
constexpr int kHalf = 4;            // tiles of half a block, which are loaded and expanded together
constexpr int kSoftWarps = 8, kDqWarps = 16;
// Warps: the softmax first (a warp reaches the tensor-memory lanes of its number mod 4).  Of the others those
// of one scheduler (number mod 4 = 0) issue MMAs, load and expand one tile, so that the MMA warp, whose few
// instructions feed the tensor cores, shares its scheduler with little; the other three schedulers' expand.
constexpr int kMmaWarp = 8, kLoadWarp = 12, kDqLast = 20, kWarpsAll = 28;   // (the load warps: 12 and 16)
constexpr int kThreads = 32 * kWarpsAll;
__device__ __forceinline__ int dq_index(int warp) {   // which expanding warp, -1: none
    if (warp < kSoftWarps) return -1;
    if (warp % 4 == 0) return warp == kDqLast ? kDqWarps - 1 : -1;
    return (warp - kSoftWarps) / 4 * 3 + warp % 4 - 1;
}
// tensor memory columns
constexpr int kTmemCols = 512;
constexpr int kColS = 0;            // 2 x 128: S; then P, each half of the keys in the first 32 columns of its 64
constexpr int kColO = 256;          // D
constexpr int kColQ = 384;          // D / 2
constexpr int kColZ = 448;          // 8 (group sums of q), 32 written
static_assert(kColO + 128 <= kColQ && kColQ + 64 <= kColZ && kColZ + 32 <= kTmemCols, "tensor memory");

template <int BITS, int D>
struct PreSmem {
    using L = KvLayout<BITS, D>;
    static constexpr int kAtoms = D / 64;                        // 128-byte rows of 64 dimensions
    static constexpr int kAtom = kKeys * 128;                    // one of them for all keys of a block
    static constexpr int kKStage = 2 * kAtoms * kAtom;           // K rounded, K's rest
    static constexpr int kVAtom = D * 128;                       // [D][64 keys]
    static constexpr int kRawTile = L::kCodes + 2 * L::kMeta;    // a tile's keys (or values): codes, S, Z
    static constexpr int kRawStage = kHalf * kRawTile;
    static constexpr int kRawK = L::kBytes <= 2560 ? 5 : 3, kRawV = L::kBytes <= 2560 ? 4 : 2;   // half blocks in flight
    static constexpr int kK = 0;
    static constexpr int kZ = kK + 2 * kKStage;                  // Z of stage b in chunk 2 b of each key's row
    static constexpr int kV = kZ + kAtom;
    static constexpr int kRawOff = kV + 2 * kVAtom;
    static constexpr int kMl = kRawOff + (kRawK + kRawV) * kRawStage;       // [2 halves][rows] maxima, then sums
    static constexpr int kF = kMl + 2 * kRows * 4;               // [rows] score factors
    static constexpr int kBars = kF + kRows * 4;
    static constexpr int kNumBars = 2 * (kRawK + kRawV) + 2 * 3 + 3;
    static constexpr int kSize = 1024 + kBars + 8 * kNumBars;
    static_assert(kSize <= 227 * 1024 && kBars % 8 == 0 && kRawOff % 128 == 0 && kRawStage % 16 == 0, "shared memory");
};

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }   // the softmax warps
// Whether any thread of a row's two warps says so (and a barrier of the two).
__device__ __forceinline__ bool pair_any(int pair, bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)mine), "r"(2 + pair)
        : "memory");
    return any != 0;
}
template <int BITS, int D, class T>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ AttnParams P) {
    using L = KvLayout<BITS, D>;
    using M = PreSmem<BITS, D>;
    constexpr int G = D / 32, kRawAll = M::kRawK + M::kRawV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // (the swizzle's 1024-byte atoms)
    float* ml = reinterpret_cast<float*>(base + M::kMl);
    float* factors = reinterpret_cast<float*>(base + M::kF);
    __shared__ uint32_t s_tmem;
    __shared__ volatile uint32_t s_there[2][16];   // a half block's tiles in the cache, keys' and values' (no role is 16 ahead of another)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const uint32_t bars = smem_u32(base + M::kBars);
    const uint32_t raw_full = bars, raw_empty = raw_full + 8 * kRawAll, k_full = raw_empty + 8 * kRawAll, s_full = k_full + 16;
    const uint32_t p_full = s_full + 16, v_full = p_full + 16, o_done = v_full + 8, q_full = o_done + 8;
    if (tid == 0) {
        for (int i = 0; i < kRawAll; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, kHalf);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full + 8 * b, 2 * kHalf);
            mbar_init(s_full + 8 * b, 1);
            mbar_init(p_full + 8 * b, kSoftWarps);
        }
        mbar_init(v_full, 2 * kHalf);
        mbar_init(o_done, 1);
        mbar_init(q_full, 4);
        fence_mbar_init();
    }
    // (the odd chunks of the Z rows multiply nothing: zero for good)
    for (int i = tid; i < M::kAtom / 16; i += kThreads) sts128(base + M::kZ + 16 * i, 0, 0, 0, 0);
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
    const int c = blockIdx.x;
    const Shares shares(P.pre_total, gridDim.x);
    const int g0 = prefix_block_at(each, shares.first(c)), g1 = prefix_block_at(each, shares.first(c + 1));
    const int blocks = g1 - g0;        // (none: nothing to do, and the second run expects nothing)
    int own_abort = 0;
    auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait_bounded(bar, parity & 1u, &own_abort, P.status); };

    if (warp == kLoadWarp || warp == kLoadWarp + 4) {
        // ---------------------------------------------------------------- keys' or values' bytes into their ring
        const int what = warp != kLoadWarp, ring = what ? M::kRawV : M::kRawK, first = what ? M::kRawK : 0;
        const uint32_t full = raw_full + 8 * first, empty = raw_empty + 8 * first;
        const uint32_t dst0 = smem_u32(base + M::kRawOff + first * M::kRawStage);
        const uint8_t* src = nullptr;
        int s = 0, turn = -1;
        for (int i = 0; i < 2 * blocks; ++i) {   // half blocks
            if (i % 8 == 0) {                    // addresses of four blocks' tiles, one per lane
                const int gb = g0 + (i + lane / kHalf) / 2;
                src = nullptr;
                if (gb < g1) {
                    const int unit = gb / each, head = unit / P.row_tiles;
                    const int tile = (gb - unit * each) * 2 * kHalf + lane % (2 * kHalf);
                    if (tile * kKvTile < P.max_len) {
                        const int pi = tile / P.cache.tiles_per_page, page = P.block_table[pi];
                        if (page < 0 || page >= P.cache.num_pages) atomicOr(P.status, kStatusIndex);
                        else
                            src = P.cache.pages + (((int64_t)page * P.cache.kv_heads + head) * P.cache.tiles_per_page +
                                                   (tile - pi * P.cache.tiles_per_page)) * (int64_t)L::kBytes;
                    }
                }
            }
            if (turn >= 0) wait(empty + 8 * s, turn);
            __syncwarp();
            const uint32_t there = (__ballot_sync(0xffffffffu, src != nullptr) >> (i % 8 * kHalf)) & ((1u << kHalf) - 1u);
            if (lane == 0) {
                s_there[what][i & 15] = there;
                if (there) mbar_arrive_expect_tx(full + 8 * s, __popc(there) * M::kRawTile);
                else mbar_arrive(full + 8 * s);
            }
            __syncwarp();
            if (lane / kHalf == i % 8 && src) {
                const uint32_t dst = dst0 + s * M::kRawStage + lane % kHalf * M::kRawTile;
                bulk_load(dst, src + (what ? L::kVc : 0), L::kCodes, full + 8 * s);
                bulk_load(dst + L::kCodes, src + (what ? L::kVs : L::kKs), 2 * L::kMeta, full + 8 * s);
            }
            if (++s == ring) s = 0, ++turn;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- all MMAs, one thread
        constexpr uint32_t idS = idesc_f16(false, kRows, kKeys), idO = idesc_f16(false, kRows, D);
        // (descriptors count 16-byte units from their first: a constant each)
        const uint64_t kd = smem_desc_sw128(smem_u32(base + M::kK)), zd = smem_desc_sw128(smem_u32(base + M::kZ));
        const uint64_t vd = smem_desc_sw128(smem_u32(base + M::kV));
        auto scores = [&](int i) {
            const int b = i & 1;
            const uint32_t d = tmem + kColS + kKeys * b;
            const uint64_t k = kd + (b ? M::kKStage / 16 : 0);
            wait(k_full + 8 * b, i >> 1);
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int st = 0; st < D / 16; ++st)
                        tc_mma_f16_ts(d, tmem + kColQ + 8 * st, k + ((part * M::kAtoms + st / 4) * M::kAtom + 32 * (st % 4)) / 16, idS,
                                      (part | st) != 0);
                tc_mma_f16_ts(d, tmem + kColZ, zd + 2 * b, idS, 1);
                tc_commit(s_full + 8 * b);
            }
            __syncwarp();
        };
        int done = 0;   // blocks of earlier units
        for (int u = 0; done < blocks; ++u) {
            const int unit = (g0 + done) / each, nb = min((unit + 1) * each, g1) - (g0 + done);
            wait(q_full, u);
            tc_fence_after();
            scores(done);
            for (int j = 0; j < nb; ++j) {
                const int i = done + j, b = i & 1;
                if (j + 1 < nb) scores(i + 1);
                wait(v_full, i);
                wait(p_full + 8 * b, i >> 1);
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int st = 0; st < kKeys / 16; ++st)
                        tc_mma_f16_ts(tmem + kColO, tmem + kColS + kKeys * b + (st / 4) * 64 + 8 * (st % 4),
                                      vd + ((st / 4) * M::kVAtom + 32 * (st % 4)) / 16, idO, j != 0 || st != 0);
                    tc_commit(o_done);
                }
                __syncwarp();
            }
            done += nb;
        }
        __syncwarp();
    } else if (dq_index(warp) >= 0) {
        // ---------------------------------------------------------------- codes to operands
        const int w = dq_index(warp), tile_no = w % kHalf, half = w / kHalf & 1;   // this warp's tile of every block
        const bool keys = w < 2 * kHalf;
        const int ring = keys ? M::kRawK : M::kRawV, first = keys ? 0 : M::kRawK, no = half * kHalf + tile_no;
        const uint8_t* raw = base + M::kRawOff + first * M::kRawStage + tile_no * M::kRawTile;
        int s = half % ring, turn = half / ring;   // half block 2 i + half in stage (2 i + half) % ring
        for (int i = 0; i < blocks; ++i) {
            const int b = i & 1, gb = g0 + i, kb = gb - gb / each * each;
            wait(raw_full + 8 * (first + s), turn);
            // the stage's last MMAs have read it
            if (keys && i >= 2) wait(s_full + 8 * b, (i >> 1) - 1);
            if (!keys && i >= 1) wait(o_done, i - 1);
            const uint8_t* tile = raw + s * M::kRawStage;
            const int left = s_there[keys ? 0 : 1][(2 * i + half) & 15] >> tile_no & 1u ? P.max_len - kb * kKeys - no * kKvTile : 0;
            if (keys) expand_keys<BITS, D>(tile, tile + L::kCodes, base + M::kK + b * M::kKStage, base + M::kZ, 2 * b, no, left, lane);
            else expand_values<BITS, D>(tile, tile + L::kCodes, base + M::kV + half * M::kVAtom, tile_no, left, lane);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(keys ? k_full + 8 * b : v_full);
                mbar_arrive(raw_empty + 8 * (first + s));
            }
            s += 2;
            if (s >= ring) s -= ring, ++turn;
        }
    } else if (warp < kSoftWarps) {
        // ---------------------------------------------------------------- softmax: two threads per row
        const int half = warp >> 2, r = 32 * (warp & 3) + lane;        // keys 64 half .. + 63 of a block
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        int done = 0;
        for (int u = 0; done < blocks; ++u) {
            const int unit = (g0 + done) / each, us = unit * each, nb = min(us + each, g1) - (g0 + done);
            const int head = unit / P.row_tiles, rt = unit - head * P.row_tiles, rows = min(kRows, P.all_rows - rt * kRows);
            if (half == 0) {
                // Q, scaled by a power of two into [2^9, 2^10), its columns in the order of K's rows
                float top = 0.f;
                const int row = rt * kRows + r, bt = row / P.group;
                const uint16_t* src = static_cast<const uint16_t*>(P.q) + bt * P.q_stride + (int64_t)(head * P.group + (row - bt * P.group)) * D;
                const bool live = r < rows;
#pragma unroll 8
                for (int k = 0; k < D / 8; ++k) {
                    const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(elem_to_float<T>((uint16_t)(w[e >> 1] >> (16 * (e & 1))))));
                }
                int e = top > 0.f ? 9 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
                e = min(max(e, -120), 120);
                const float up = pow2i(e);
                factors[r] = P.scale_log2 * pow2i(-e);
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
            float m = -INFINITY, l = 0.f, ref = 0.f;
            for (int j = 0; j < nb; ++j) {
                const int i = done + j, b = i & 1;
                wait(s_full + 8 * b, i >> 1);
                tc_fence_after();
                const uint32_t col = lanes + kColS + kKeys * b + 64 * half;
                const int left = P.max_len - (g0 + i - us) * kKeys - 64 * half;   // keys of the prefix from this half's first on
                const uint32_t there = s_there[0][(2 * i + half) & 15];
                const bool some = left < 64 || there != (1u << kHalf) - 1u;
                // 32 scores at a time, read twice (for the maximum and for P): registers are what 28 warps leave
                auto load = [&](int h, float (&x)[32]) {
                    tmem_ld32(col + 32 * h, reinterpret_cast<uint32_t(&)[32]>(x));
                    if (some) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * h + k >= left || !(there >> ((32 * h + k) / kKvTile) & 1u)) x[k] = -INFINITY;
                    }
                };
                float mx = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[32];
                    load(h, x);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) mx = fmaxf(fmaxf(mx, x[k]), x[k + 1]);
                }
                mx *= f;
                if (pair_any(warp & 3, mx > m + kTau)) {
                    ml[half * kRows + r] = mx;
                    pair_any(warp & 3, false);
                    mx = fmaxf(mx, ml[(half ^ 1) * kRows + r]);
                    const float now = mx > m + kTau ? mx : m, a = m == now ? 1.f : ex2(m - now);
                    if (j > 0 && __any_sync(0xffffffffu, m != now)) {   // each thread its half of O's dimensions
                        wait(o_done, i - 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
                            uint32_t o[32];
                            tmem_ld32(lanes + kColO + d, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                            tmem_st32(lanes + kColO + d, o);
                        }
                    }
                    l *= a;
                    m = now;
                    ref = now == -INFINITY ? 0.f : now - kPBits;
                }
                // The O before, whether or not a reference moved: the wait for the unit's last O would otherwise take the
                // end of the phase before the last for it.  (P's MMAs come after that O's in any case; waited for here and
                // not after P: 118.8 -> 116.6 us.)
                if (i > 0) wait(o_done, i - 1);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[32];
                    load(h, x);
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 y = fma2(make_float2(x[k], x[k + 1]), make_float2(f, f), make_float2(-ref, -ref));
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum = add2(sum, e);
                        p[k / 2] = pack_half2_rn(e.x, e.y);
                    }
                    tmem_st16(col + 16 * h, p);   // (over scores that have been read)
                }
                l += sum.x + sum.y;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * b);
            }

            // ---- the unit's rows: each thread half of its row's dimensions ----
            soft_sync();   // (the maxima's last readers are done)
            ml[half * kRows + r] = l;
            soft_sync();
            l = ml[r] + ml[kRows + r];
            wait(o_done, done + nb - 1);
            tc_fence_after();
            // into this block's slot of the unit: the second run joins the slots
            float* slot = P.pre_o + (int64_t)(c * P.pre_slots + prefix_slot(shares, each, c, unit)) * (kRows * (D + 2));
            if (half == 0 && r < rows) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(m, l);
#pragma unroll 1
            for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
                uint32_t a[32];
                tmem_ld32(lanes + kColO + d, a);
                if (r < rows) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4*>(slot + r * D + d + k) = make_uint4(a[k], a[k + 1], a[k + 2], a[k + 3]);
                }
            }
            tc_fence_before();
            soft_sync();   // both halves are done with O, the factors and the sums
            done += nb;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int BITS, int D, class T>
lq_status run(lq_handle h, const AttnParams& P, cudaStream_t stream) {
    using M = PreSmem<BITS, D>;
    static std::mutex mu;
    static bool ready[kMaxDevices] = {};   // the shared-memory attribute is set
    if (h->device < 0 || h->device >= kMaxDevices || M::kSize > h->max_smem_optin) return LQ_ERR_UNSUPPORTED;
    {
        const std::lock_guard<std::mutex> lock(mu);
        if (!ready[h->device]) {
            if (cudaFuncSetAttribute(prefix_kernel<BITS, D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kSize) != cudaSuccess)
                return LQ_ERR_CUDA;
            ready[h->device] = true;
        }
    }
    return launch_overlapped(prefix_kernel<BITS, D, T>, P.pre_blocks, kThreads, M::kSize, stream, P);
}

// Places of all units' key blocks, with each unit's fixed cost before them, which the thread blocks share.
int64_t key_places(int kv_heads, int all_rows, int prefix_len) {
    return (int64_t)kv_heads * ((all_rows + kRows - 1) / kRows) * ((prefix_len + kKeys - 1) / kKeys + kPreUnitCost);
}

}  // namespace

// Taken from 17 rows per kv head (where the other kernel reads the prefix once per 16 rows) and 385 shared tokens
// on (where the other cuts a unit into pieces and joins them).  Measured (whole call, 128 dimensions, 4 bits, one own token;
// this kernel and the other, us) over 256 / 384 / 1000 / 4000 / 16000 tokens, 8 kv heads unless it says 32:
//     17 rows         18.5, 19.5 / 18.6, 20.4 / 19.4, 24.6 / 22.8, 25.7 / 30.9, 34.9
//     17 rows, 32     20.9, 19.9 / 21.4, 21.0 / 23.3, 28.8 / 32.4, 37.0 / 66.9, 74.7
//     136 of group 8  22.7, 20.3 / 22.8, 20.9 / 25.0, 30.0 / 29.9, 39.3 / 47.4, 78.0
//     512 of group 8  27.4, 31.1 / 27.3, 37.5 / 29.5, 46.1 / 38.4, 79.4 / 72.5, 218
//     8192 of group 8 208, 254 / 214, 278 / 256, 406 / 400, 934
//     1024 of group 1 129, 126 / 131, 130 / 137, 145 / 155, 209 / 221, 479
//     1024, 32        478, 479 / 483, 495 / 506, 557 / 584, 825
// So up to 384 tokens the other one is as good or better up to 200 rows, and gives away up to a quarter from 512 rows of
// wide groups on.  Earlier figures for 16 rows: 15.0, 20.2 over 1000 tokens with 8 heads, but 29.3, 27.9 over 16000 and 64.9,
// 51.5 with 32 heads.  8 bits: the same within 10 %.
size_t prefix_tc_bytes(lq_handle h, int kv_heads, int all_rows, int prefix_len, int D) {
    const int64_t n = key_places(kv_heads, all_rows, prefix_len);
    if (all_rows <= 16 || prefix_len <= 384 || n > 0x7fffffffLL) return 0;
    const int blocks = (int)std::min<int64_t>(h->num_sms, n);
    return (size_t)blocks * prefix_slots((prefix_len + kKeys - 1) / kKeys, (int)n, blocks) * kRows * (D + 2) * sizeof(float);
}

lq_status launch_prefix_tc(lq_handle h, AttnParams& P, int bits, int D, bool bf16, char* scratch, cudaStream_t stream) {
    P.pre_o = reinterpret_cast<float*>(scratch);
    P.pre_rows = kRows;
    P.row_tiles = P.pre_tiles = (P.all_rows + kRows - 1) / kRows;
    P.pre_each = (P.max_len + kKeys - 1) / kKeys;
    P.pre_total = (int)key_places(P.cache.kv_heads, P.all_rows, P.max_len);
    P.pre_blocks = std::min(h->num_sms, P.pre_total);
    P.pre_slots = prefix_slots(P.pre_each, P.pre_total, P.pre_blocks);
    if (D == 128) {
        if (bits == 4) return bf16 ? run<4, 128, __nv_bfloat16>(h, P, stream) : run<4, 128, __half>(h, P, stream);
        return bf16 ? run<8, 128, __nv_bfloat16>(h, P, stream) : run<8, 128, __half>(h, P, stream);
    }
    if (bits == 4) return bf16 ? run<4, 64, __nv_bfloat16>(h, P, stream) : run<4, 64, __half>(h, P, stream);
    return bf16 ? run<8, 64, __nv_bfloat16>(h, P, stream) : run<8, 64, __half>(h, P, stream);
}

}  // namespace lq
