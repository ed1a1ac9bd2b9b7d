// The low-bit KV cache: where a tile keeps its codes, scales and offsets, and the register
// moves between a row of 8 dimensions per lane and the tile's words.
//
// A tile holds 16 consecutive tokens of one kv head.  Its codes lie in the order in which a
// warp's m16n8k16 fragments take them (lane = 4 n + t, n 0..7, t 0..3), each lane's words as
// 16-byte chunks [chunk][lane][16 B], so that a warp reads a tile with plain conflict-free
// 16-byte shared-memory loads and expands codes to operands with masks and shifts only:
//   keys    word hf * WK + w of lane (n, t): token n + 8 hf;
//           4-bit: w = g, nibble e is dimension 32 g + 8 t + e;
//           8-bit: w = 2 g + u, byte e is dimension 32 g + 8 t + 4 u + e.
//   values  word j * WV + wi of lane (n, t): token 2 t + (j & 1) + 8 (j >> 1);
//           element e is dimension 8 (e * WV + wi) + n.
// then keys' S [16][G], keys' Z [16][G], values' S [G][16], values' Z [G][16] (binary16), the
// values' tokens in the order kv_vmeta_pos, which puts the four of a lane side by side.
#pragma once

#include <stdint.h>

#include "lq_common.cuh"

namespace lq {

constexpr int kKvTile = 16;    // tokens of a tile
constexpr int kKvGroup = 32;   // dimensions that share S and Z

template <int BITS, int D>
struct KvLayout {
    static constexpr int G = D / kKvGroup;
    static constexpr int kPer = 32 / BITS;               // codes of a word
    static constexpr int WK = D / (4 * kPer);            // key words of a lane and token
    static constexpr int WV = D / (8 * kPer);            // value words of a lane and token
    static constexpr int kChunks = WK / 2;               // 16-byte chunks of a lane (keys; values alike)
    static constexpr int kCodes = kKvTile * D * BITS / 8;
    static constexpr int kMeta = kKvTile * G * 2;
    static constexpr int kVc = kCodes, kKs = 2 * kCodes, kKz = kKs + kMeta, kVs = kKz + kMeta, kVz = kVs + kMeta;
    static constexpr int kBytes = kVz + kMeta;
    static_assert(2 * WK == 4 * WV && 2 * WK % 4 == 0 && kBytes % 16 == 0, "tile layout");
};

__host__ __device__ constexpr int kv_tile_bytes(int bits, int D) {
    return kKvTile * (2 * D * bits / 8 + 2 * (D / kKvGroup) * 4);
}

// Byte of word `q` of a lane inside a code region.
__device__ __forceinline__ int kv_word_at(int lane, int q) { return (q >> 2) * 512 + lane * 16 + (q & 3) * 4; }
// Place of a token of the tile in the values' S and Z rows.
__device__ __forceinline__ int kv_vmeta_pos(int tok) { return 4 * ((tok & 7) >> 1) + (tok & 1) + 2 * (tok >> 3); }

// 8 x 8 nibbles over eight lanes `step` apart (e: this lane's index among them): lane e gives
// its word's nibble i to lane i, and gets nibble e of every lane's word in lane order.
__device__ __forceinline__ uint32_t kv_transpose_nibbles(uint32_t w, int e, int step) {
#pragma unroll
    for (int s = 4; s >= 1; s >>= 1) {
        const uint32_t low = s == 4 ? 0x0000FFFFu : (s == 2 ? 0x00FF00FFu : 0x0F0F0F0Fu);
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w, s * step);
        w = (e & s) ? ((o >> (4 * s)) & low) | (w & ~low) : (w & low) | ((o & low) << (4 * s));
    }
    return w;
}
// 4 x 4 bytes over four lanes `step` apart.
__device__ __forceinline__ uint32_t kv_transpose_bytes(uint32_t w, int e, int step) {
#pragma unroll
    for (int s = 2; s >= 1; s >>= 1) {
        const uint32_t low = s == 2 ? 0x0000FFFFu : 0x00FF00FFu;
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w, s * step);
        w = (e & s) ? ((o >> (8 * s)) & low) | (w & ~low) : (w & low) | ((o & low) << (8 * s));
    }
    return w;
}

// The cache as the kernels see it.
struct KvView {
    uint8_t* pages;
    int64_t num_pages;
    int page_size, kv_heads, tiles_per_page;
};

}  // namespace lq
