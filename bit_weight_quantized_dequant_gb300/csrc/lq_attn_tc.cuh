// What the dense attention kernels (lq_attn_prefix.cu, lq_attn_chunk.cu) share: cached codes becoming binary16 operands of
// the tensor-memory tensor cores, in shared memory with the 128-byte swizzle.
#pragma once

#include "lq_attn.cuh"
#include "lq_tcgen05.cuh"

namespace lq {

constexpr int kTcKeys = 128;        // keys of a block
// A K-major operand of D columns and KEYS rows: rows of 64 values (128 bytes), KEYS of them an atom.
template <int D, int KEYS = kTcKeys>
struct TcOperand {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtom = KEYS * 128;
};

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return reinterpret_cast<__half2&>(v); }
__device__ __forceinline__ uint32_t as_bits(__half2 v) { return reinterpret_cast<uint32_t&>(v); }
// Two fp32 values at a time.
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
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint8_t* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

// A masked code as a whole number: it stands in the low bits of 1024 (or, 4 bits up, of 64).
__device__ __forceinline__ __half2 less_1024(uint32_t v) { return __hadd2(as_half2(v | 0x64006400u), as_half2(0xe400e400u)); }
__device__ __forceinline__ __half2 less_64(uint32_t v) { return __hadd2(as_half2(v | 0x54005400u), as_half2(0xd400d400u)); }

// Whole numbers (binary16 pairs) of a word's codes: 4-bit r = 0..3: nibbles (r, r + 4); 8-bit
// r = 0, 1: bytes (r, r + 2).
template <int BITS>
__device__ __forceinline__ __half2 code_pair(uint32_t w, int r) {
    if (BITS == 4) {
        const uint32_t y = r & 2 ? w >> 8 : w;
        return r & 1 ? less_64(y & 0x00f000f0u) : less_1024(y & 0x000f000fu);
    }
    return __hadd2(as_half2(prmt(w, 0x64646464u, r ? 0x4341 : 0x4240)), as_half2(0xe400e400u));
}

// Not past the end of binary16's range (NaN stays).
__device__ __forceinline__ __half2 clamp_top(__half2 v) { return __hmin2_nan(v, __float2half2_rn(65504.f)); }
template <bool CLAMP>
__device__ __forceinline__ __half2 clamped(__half2 v) { return CLAMP ? clamp_top(v) : v; }

// Keys of one tile: [token][dims] rows of the K stage, in the order of the words' pairs (Q's columns
// follow it), and Z.  left: tokens of the prefix from the tile's first on.
template <int BITS, int D, int KEYS = kTcKeys, bool CLAMP = true>
__device__ __forceinline__ void expand_keys(const uint8_t* tile, const uint8_t* meta, uint8_t* stage, uint8_t* zs, int zchunk, int tile_no, int left, int lane) {
    using L = KvLayout<BITS, D>;
    using M = TcOperand<D, KEYS>;
    constexpr int G = D / 32, WK = L::WK, U = WK / G;   // U words of a group (1 or 2)
    const int n = lane >> 2, t = lane & 3, odd = n & 1;
    // Odd tokens take their groups two by two in the other order (below: group st ^ odd at step st), so that
    // eight lanes write to eight places.
    const int even_at = ((4 * odd + t) ^ n) << 4, odd_at = ((4 * (odd ^ 1) + t) ^ n) << 4;
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
        uint32_t s[G / 2], z[G / 2];                             // groups (2 i, 2 i + 1)
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
            const uint32_t v = lds32(meta + tok * G * 2 + 4 * i) & keep;
            s[i] = odd ? prmt(v, v, 0x1032) : v;
            z[i] = lds32(meta + L::kMeta + tok * G * 2 + 4 * i) & keep;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t x = kw[U * 2 * i + u], y = kw[U * (2 * i + 1) + u];
                kw[U * 2 * i + u] = odd ? y : x;
                kw[U * (2 * i + 1) + u] = odd ? x : y;
            }
        }
        uint8_t* base = stage + row * 128;
#pragma unroll
        for (int st = 0; st < G; ++st) {
            const __half2 s2 = st & 1 ? __high2half2(as_half2(s[st >> 1])) : __low2half2(as_half2(s[st >> 1]));
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 c = code_pair<BITS>(kw[U * st + i / (4 / U)], i % (4 / U)), p = clamped<CLAMP>(__hmul2(c, s2));
                hi[i] = as_bits(p);
                lo[i] = as_bits(clamped<CLAMP>(__hfma2(c, s2, __hneg2(p))));     // c S - p, exactly (unless p was clamped)
            }
            uint8_t* at = base + (st & 1 ? odd_at : even_at) + (st >> 1) * M::kAtom;
            sts128(at, hi[0], hi[1], hi[2], hi[3]);
            sts128(at + M::kAtoms * M::kAtom, lo[0], lo[1], lo[2], lo[3]);
        }
        if (t == 0) {   // Z against both terms of the group sums
            uint8_t* at = zs + row * 128 + ((zchunk ^ n) << 4);
            if (G == 4) sts128(at, z[0], z[G / 2 - 1], z[0], z[G / 2 - 1]);
            else sts128(at, z[0], z[0], 0u, 0u);
        }
    }
}

// Values of one tile: [dimension][keys] rows of the V stage, two keys per word.  PARTS = 2: only half of the dimensions, those
// whose codes lie in the lower (part 0) or upper halves of the words.
template <int BITS, int D, int PARTS = 1, bool CLAMP = true>
__device__ __forceinline__ void expand_values(const uint8_t* tile, const uint8_t* meta, uint8_t* stage, int tile_no, int left, int lane, int part = 0) {
    using L = KvLayout<BITS, D>;
    constexpr int G = D / 32 / PARTS, WV = L::WV, kPer = 32 / BITS;
    const int n = lane >> 2, t = lane & 3;
    alignas(16) uint32_t vw[4 * WV];
#pragma unroll
    for (int c = 0; c < L::kChunks; ++c)
        *reinterpret_cast<uint4*>(vw + 4 * c) = lds128(tile + 512 * c + 16 * lane);
    const uint32_t keep[2] = {(2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u),
                              (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u)};
    uint8_t* at[2] = {stage + n * 128 + (((2 * tile_no) ^ n) << 4) + 4 * t, stage + n * 128 + (((2 * tile_no + 1) ^ n) << 4) + 4 * t};
    meta += part * G * 32;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint2 sv = lds64(meta + g * 32 + 8 * t), zv = lds64(meta + L::kMeta + g * 32 + 8 * t);
        const uint32_t s[2] = {sv.x & keep[0], sv.y & keep[1]}, z[2] = {zv.x & keep[0], zv.y & keep[1]};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int slab = 4 * g + k, wi = slab % WV, e = slab / WV;   // dimension 8 slab + n (of the part's)
            const uint32_t halves = PARTS == 2 ? (part ? 0x7632 : 0x5410) : e < kPer / 2 ? 0x5410 : 0x7632;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t wa = vw[2 * half * WV + wi], wb = vw[(2 * half + 1) * WV + wi];
                const uint32_t y = prmt(wa, wb, halves);
                __half2 c;
                if (BITS == 4) {
                    const uint32_t w = (e & 2) ? y >> 8 : y;
                    c = (e & 1) ? less_64(w & 0x00f000f0u) : less_1024(w & 0x000f000fu);
                } else {
                    const uint32_t w = (e & 1) ? y >> 8 : y;
                    c = less_1024(w & 0x00ff00ffu);
                }
                const __half2 v = clamped<CLAMP>(__hfma2(c, as_half2(s[half]), as_half2(z[half])));   // (S rounded up may pass it)
                *reinterpret_cast<uint32_t*>(at[half] + slab * 1024) = as_bits(v);
            }
        }
    }
}

}  // namespace lq
