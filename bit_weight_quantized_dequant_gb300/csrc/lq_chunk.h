// What the chunk attention kernel's blocks share out: tiles of a request's new rows, and the key blocks that each of them
// visits.  Whole-number arithmetic of the host and the device alike, so that it can be walked through without a GPU.
#pragma once

#include <stdint.h>

#include "lq_share.h"

namespace lq {

constexpr int kChunkKeys = 128;      // keys of a block
// What a unit counts in its key blocks besides them.  (It costs a pair about seven, but what is cut finer ends more evenly: with 3, 6 and 10
// windowed chunks of 3 requests 35.8, 39.9 and 39.2 us, 12 ragged requests 441, 446 and 475.)
constexpr int kChunkUnitCost = 3;

// Tile `rt` (of `tile_rows` rows) of a request of `len` tokens of which `fresh` are new: its rows are (new token, query head of
// the group), tokens slower.  window 0: none.
struct ChunkTile {
    int p0, p1;        // positions of its first and last row (below 0: it sees nothing)
    int lowest;        // the first token that a row's window holds
    int sunk, gap;     // key blocks that hold sinks only, and those left out behind them
    int blocks;        // key blocks that it visits, 1 at least
    LQ_HD ChunkTile(int len, int fresh, int group, int window, int sinks, int tile_rows, int rt) {
        const unsigned r0 = (unsigned)rt * tile_rows, rows = (unsigned)fresh * group, all = r0 + tile_rows;   // (below 2^31)
        p0 = len - fresh + (int)(r0 / (unsigned)group);
        p1 = len - fresh + (int)(((all < rows ? all : rows) - 1) / (unsigned)group);
        lowest = window > 0 && p0 >= window ? p0 - window + 1 : 0;
        const int from = lowest / kChunkKeys, end = (p1 < 0 ? 0 : p1 / kChunkKeys + 1);
        const int s = (int)(((unsigned)sinks + kChunkKeys - 1) / kChunkKeys);
        sunk = s < from ? s : from;
        gap = from - sunk;
        blocks = end - gap > 1 ? end - gap : 1;
    }
    LQ_HD int block(int i) const { return i < sunk ? i : i + gap; }      // number of the i-th block visited
    // whether every row sees all of key block kb
    LQ_HD bool whole(int kb, int window, int sinks) const {
        const int64_t first = (int64_t)kb * kChunkKeys, last = first + kChunkKeys - 1;
        return last <= p0 && (window <= 0 || first > (int64_t)p1 - window || last < sinks);
    }
};

LQ_HD int chunk_tiles(int fresh, int group, int tile_rows) { return (int)(((unsigned)fresh * group + tile_rows - 1) / (unsigned)tile_rows); }

// n things shared out to c parties in order, as Shares, past 32 bits.
struct WideShares {
    int64_t q, rem;
    LQ_HD WideShares(int64_t n, int c) : q(n / c), rem(n - q * c) {}
    LQ_HD int64_t first(int k) const { return q * k + (k < rem ? k : rem); }
    LQ_HD int of(int64_t i) const {
        const int64_t more = rem * (q + 1);
        return (int)(i < more ? i / (q + 1) : rem + (i - more) / q);
    }
};

}  // namespace lq
