// Attention of chunks of new tokens over the low-bit KV cache, on the tensor-memory tensor cores.
//
// A unit is 256 rows of one kv head of one request (rows are (new token, query head of the group), tokens slower) and the
// blocks of 128 keys that they see.  A pair of CTAs takes it, 128 rows in each one's tensor memory:
//   S [rows][128 keys] = Q K^T     Q in tensor memory, K in shared memory
//   P = 2^(S f - m)                S read from and P written to tensor memory
//   O [rows][D]       += P V       P in tensor memory, V [D][128 keys] in shared memory
// by tcgen05.mma.cta_group::2 (M 256, binary16 operands, fp32 sums), of whose other operand each CTA holds half: the keys of
// half a block, the values' half of the dimensions.  So each code is expanded once for 256 rows; one CTA with 128 rows
// spent its issue slots on that (2048 tokens at the end of 32 Ki, 64 query heads over 8, 128 dimensions, 4 bits, bf16: 3582 us,
// the pair 2985 with all else as it was).
//
// Operands and precision are those of lq_attn_prefix.cu: K's code part as two binary16 terms and its offset part as one more MMA
// of 16 columns, so that scores keep fp32 precision; V and P rounded to binary16.  Binary16 outputs, whose own rounding is no
// coarser, multiply what P's left out too (error of windowed chunks 3.2e-4 -> 2.9e-4, where the output's rounding alone is
// 2.1e-4; 37 -> 42 us).  Terms past the end of binary16's range are clamped, in tiles whose S or Z say that there may be some.
//
// What is this kernel's own:
//   - Every request has rows, pages and a length of its own, read on the device.  All units' key blocks form one sequence,
//     each unit counted with its fixed cost, which the pairs share evenly (lq_chunk.h); a unit that is cut leaves partial
//     sums in the workspace, and the last of its pairs to arrive joins them in order (results repeat bit for bit).
//   - A row sees the tokens up to its own, and with a window the last of them and the sinks.  Blocks that no row of the unit
//     sees are not visited; in one that not every row sees whole, scores are masked by two bounds per row.
//   - A P of 0 times a cached NaN is NaN, so a value group (token and 32 dimensions) whose S or Z is no number counts as 0
//     in the product, and rows that do see it get NaN in those dimensions at the unit's end.  So does, in a tile whose S or Z are
//     large or no numbers, every value between the sinks and the windows, which may be anything and is nobody's.
//
// Roles (23 warps of 24): two load keys' and values' bytes by bulk copies, each into a ring of its own; one issues the MMAs (in
// the even CTA); twelve expand codes, a 16-token tile each, four this CTA's keys, eight its half of all values' dimensions;
// eight do the softmax, two threads per row with half of the keys each.  S and the stages of K and V are double: the next
// block's scores are computed while this one's softmax runs.  All MMAs come from one thread and end in its order, so few
// barriers suffice: K full, scores there (which frees K's stage and says that the product of the block before the last is done),
// P full, V full, O done.  A wait tells a barrier's phases apart by their parity alone: every role waits for each phase
// in turn, or at a point where the one before is known to have ended.  Every wait on a barrier in memory is bounded; a role whose
// wait ran out goes on with what is there, so every loop ends, and the status word reports it.
//
// The steps from there, the same call: the MMA warp on a scheduler without expanding warps and its operands in uniform registers
// (one elected lane) 2427 us; scores held in registers (read once), P by the reference so far while the two halves of a row find out
// whether it has to move, which a limit of 2^7 makes rare, and clamps only where needed 2176; maximum and P of a block in one go 2027
// (1050 TFLOP/s, 55 % of a library product's rate).  A unit's queries are put in place, and the scores begin, before the rows of the unit
// before are written: a prompt of 2048 tokens of 40 heads 110 -> 98 us, 65 tokens at 365 17.9 -> 12.8.  Measured and not kept: a thread per row and every other
// block for each half of the softmax warps (2527), a whole row's check by the sum of its P (2286), the next block's scores loaded ahead
// (spills: 2900), queries by bulk copies one unit ahead, and rows written from shared memory by bulk copies (65 tokens at 365
// 13.2 -> 15.1, windowed chunks 42 -> 47), both through shared memory with a warp's accesses side by side (2048 tokens
// at the end of 32 Ki 2055 -> 2115, windowed chunks 42 -> 41),
// a longer suspension of waiting warps (no change).
//
// What bounds it now: the softmax of a block takes about 1900 cycles from its scores to its P, one block after another,
// where its 25 MMAs take 1620 (tensor pipe 58 %, issue 63 %).  That is this schedule's bound, not the hardware's: a second row
// tile's softmax could run under the first one's MMAs.  With heads of 64 dimensions two tiles' S, O and Q take 464 of tensor memory's
// 512 columns; with 128 Q would have to be the operand in shared memory (S and O alone fill 512).  Not built.  The 206 to 240 bytes a
// thread that the compiler spills are seldom touched: 0.4 % of the instructions executed are local loads and stores.

#include <algorithm>
#include <mutex>

#include "lq_attn_tc.cuh"
#include "lq_chunk.h"

namespace lq {
namespace {

struct ChunkParams {
    KvView cache;
    const void* q;
    void* out;
    float* lse;
    int64_t q_stride, out_stride, bt_stride;
    const int32_t *block_table, *lens, *starts;
    int requests, tokens, group, q_heads, max_len;
    int window, sinks;
    float scale_log2;
    float* part;           // partial sums: 2 slots per CTA
    unsigned* counters;    // one per CTA, zero between calls
    int* status;
};

constexpr int kCtas = 2;            // CTAs of a pair
constexpr int kRows = 128;          // rows of a CTA
constexpr int kKeys = kTcKeys;      // keys of a block
static_assert(kKeys == kChunkKeys, "key blocks");
constexpr int kTiles = kKeys / kKvTile;
// Blocks of which is held what values are no numbers.  It is read behind the P of two blocks later; what has this place next
// is written when the product of two blocks before its own is done, so five would do (a power of two).
constexpr int kOdd = 8;
// Warps: the softmax first (a warp reaches the tensor-memory lanes of its number mod 4).  Of the others those of one
// scheduler (number mod 4 = 0) issue MMAs and load, the other three schedulers' expand: the MMA warp's instructions, few
// and each waited for by the tensor cores, are not in line behind theirs.
constexpr int kSoftWarps = 8, kKeyWarps = 4, kValueWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 12;      // (load warps: 12 keys', 16 values')
constexpr int kWarpsAll = 24, kThreads = 32 * kWarpsAll;
__device__ __forceinline__ int dq_index(int warp) {   // which expanding warp (the first four keys'), -1: none
    return warp < kSoftWarps || warp % 4 == 0 ? -1 : (warp - kSoftWarps) / 4 * 3 + warp % 4 - 1;
}
// P = 2^kPUp p in binary16, and a row's reference moves when a score passes it by 2^kPast: P stays below 2^15, and a move,
// for which the sums so far are read and written, is rare.  (2^-33 is what a probability is off by at least.)
constexpr float kPUp = 8.f, kPast = 7.f;

// registers of a thread at launch (what its bounds give), then of the softmax's and the others'
constexpr int kRegs = 80, kSoftRegs = 112, kOtherRegs = 64;
static_assert(32 * (kSoftWarps * kSoftRegs + (kWarpsAll - kSoftWarps) * kOtherRegs) <= kThreads * kRegs, "registers");
static_assert((kWarpsAll - kSoftWarps) / 4 * 3 == kKeyWarps + kValueWarps, "expanding warps");
// tensor memory columns
constexpr int kTmemCols = 512;
constexpr int kColS = 0;            // 2 x 128: S; then P, each half of the keys in the first 32 columns of its 64 (what its rounding left out in the others)
constexpr int kColO = 256;          // D
constexpr int kColQ = 384;          // D / 2
constexpr int kColZ = 448;          // 8 (group sums of q)
static_assert(kColO + 128 <= kColQ && kColQ + 64 <= kColZ && kColZ + 8 <= kTmemCols, "tensor memory");

// Shared memory of one CTA of the pair: its half of a block's keys (rows of K) and of the dimensions (rows of V).
template <int BITS, int D>
struct ChunkSmem {
    using L = KvLayout<BITS, D>;
    static constexpr int kKeysHere = kKeys / kCtas, kTilesHere = kTiles / kCtas, kDimsHere = D / kCtas;
    static constexpr int kAtoms = TcOperand<D, kKeysHere>::kAtoms, kAtom = TcOperand<D, kKeysHere>::kAtom;
    static constexpr int kKStage = 2 * kAtoms * kAtom;           // K rounded, K's rest
    static constexpr int kVAtom = kDimsHere * 128;               // [dimensions][64 keys]
    static constexpr int kRawTile = L::kCodes + 2 * L::kMeta;    // a tile's keys (or values): codes, S, Z
    static constexpr int kRawStageK = kTilesHere * kRawTile, kRawStageV = kTiles * kRawTile;
    static constexpr int kRaw = 3;                               // blocks in flight (a fourth: 430 -> 432 us for ragged requests)
    static constexpr int kK = 0;
    static constexpr int kZ = kK + 2 * kKStage;                  // Z of stage b in chunk 2 b of each key's row
    static constexpr int kV = kZ + kAtom;                        // two stages
    static constexpr int kRawK = kV + 2 * 2 * kVAtom, kRawV = kRawK + kRaw * kRawStageK;
    static constexpr int kMl = kRawV + kRaw * kRawStageV;        // [2 halves][rows] maxima, then sums
    static constexpr int kF = kMl + 2 * kRows * 4;               // [2 halves][rows] queries' largest values
    static constexpr int kGroups = kF + 2 * kRows * 4;           // [rows] queries' group sums, their rests
    static constexpr int kBad = kGroups + kRows * 2 * (D / 32) * 2;                  // [kOdd blocks][keys] groups of a value that are no numbers
    static constexpr int kBars = kBad + kOdd * kKeys;
    static constexpr int kNumBars = 4 * kRaw + 2 * 5 + 1;
    static constexpr int kSize = 1024 + kBars + 8 * kNumBars;
    static_assert(kSize <= 226 * 1024 && kBars % 8 == 0 && kRawK % 128 == 0 && kRawTile % 16 == 0, "shared memory");
    static_assert(3 * 8 * (kMaxAttnBatch + 1) <= 2 * kKStage, "the requests' running sums lie where K will");
};

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }   // the softmax warps
// The two warps of the same rows.  (Both wait: with an arrival of its own for each direction, a warp that is ahead could arrive
// twice before the other has waited once.)
__device__ __forceinline__ void rows_sync(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory"); }

// One lane of a whole warp, which the compiler knows to be one: operands of what it issues stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// The bits below n of 32 (n of any sign).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// A place in the sequence of units: the request, the row tile, the kv head.
struct Unit {
    int b, rt, head;
};

// Requests as the kernel sees them: whatever the arrays hold, rows stay within the call's.
struct Request {
    int row0, fresh, len;
    __device__ __forceinline__ Request(const ChunkParams& P, int b) {
        row0 = min(max(P.starts[b], 0), P.tokens);
        fresh = min(max(P.starts[b + 1], row0), P.tokens) - row0;
        len = min(max(P.lens[b], 0), P.max_len);
    }
};
__device__ __forceinline__ ChunkTile tile_of(const ChunkParams& P, const Request& q, int rt) {
    return ChunkTile(q.len, q.fresh, P.group, P.window, P.sinks, kCtas * kRows, rt);
}

// A thread's row of a unit: its place in q and out, its head, its token's position.
struct Row {
    int64_t at;
    int qh, p;
    bool live;
    __device__ __forceinline__ Row(const ChunkParams& P, const Request& q, const Unit& u, int rank, int r) {
        const int row = (u.rt * kCtas + rank) * kRows + r, tok = (unsigned)row / (unsigned)P.group;
        live = row < q.fresh * P.group;
        at = (int64_t)q.row0 + tok;
        qh = u.head * P.group + (row - tok * P.group);
        p = live ? q.len - q.fresh + tok : -1;
    }
};

// A pair's share: from block `j0` of unit `first` (at `place` of the sequence) to before block `j1` of unit `last`.
struct Range {
    Unit first, last;
    int j0, j1;
    int64_t place;
    bool none;
};

// A walk over a share's units; every role has one.
struct Walk {
    const ChunkParams& P;
    Range R;
    Unit u;
    Request q;
    ChunkTile t;
    int j0, j1;          // blocks of this unit that are this pair's
    int64_t place;       // of the unit's cost, its blocks follow
    bool more;
    __device__ __forceinline__ Walk(const ChunkParams& P_, const Range& r)
        : P(P_), R(r), u(r.first), q(P_, r.first.b), t(tile_of(P_, q, r.first.rt)), place(r.place), more(!r.none) {
        j0 = r.j0;
        set_end();
    }
    __device__ __forceinline__ bool at_last() const { return u.b == R.last.b && u.rt == R.last.rt && u.head == R.last.head; }
    __device__ __forceinline__ void set_end() {
        j1 = at_last() ? R.j1 : t.blocks;
        if (j1 <= j0) more = false;
    }
    __device__ __forceinline__ void next() {
        if (at_last()) {
            more = false;
            return;
        }
        place += t.blocks + kChunkUnitCost;
        j0 = 0;
        if (++u.head == P.cache.kv_heads) {
            u.head = 0;
            if (++u.rt == chunk_tiles(q.fresh, P.group, kCtas * kRows)) {
                u.rt = 0;
                do ++u.b; while (Request(P, u.b).fresh == 0);   // (the last unit lies ahead)
                q = Request(P, u.b);
            }
            t = tile_of(P, q, u.rt);
        }
        set_end();
    }
};

// Parties that share a sequence of places: so many that none has fewer than kLeast, which costs less than joining a unit's parts.
__device__ __forceinline__ int parties(int64_t total, int C) {
    constexpr int kLeast = 2 * kChunkUnitCost;
    return total >= (int64_t)kLeast * C ? C : max(1, (int)total / kLeast);
}

// (All threads of a CTA together.)  The share of party c of C; `cum` has room for three sums of each request.
__device__ __forceinline__ Range range_of(const ChunkParams& P, int c, int C, int64_t* cum, int64_t* total_out, Range* out) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto from_of = [&](int which) { return cum + (which + 1) * (kMaxAttnBatch + 1); };   // where each request's places begin, two copies
    // places of each request
    for (int b = warp; b < P.requests; b += kWarpsAll) {
        const Request q(P, b);
        if (lane == 0 && c == 0) {
            const int a0 = P.starts[b], a1 = P.starts[b + 1];
            if (a0 < 0 || a1 < a0 || a1 > P.tokens) atomicOr(P.status, kStatusIndex);
        }
        const int tiles = chunk_tiles(q.fresh, P.group, kCtas * kRows);
        int64_t sum = 0;
        for (int rt = lane; rt < tiles; rt += 32) sum += tile_of(P, q, rt).blocks + kChunkUnitCost;
#pragma unroll
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) cum[b + 1] = sum * P.cache.kv_heads;
    }
    __syncthreads();
    if (warp < 2) {        // the first place by one warp, the last by another
        int64_t base = 0;
        for (int b0 = 0; b0 < P.requests; b0 += 32) {
            const int64_t mine = b0 + lane < P.requests ? cum[b0 + lane + 1] : 0;
            int64_t v = mine;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, v, s);
                if (lane >= s) v += x;
            }
            if (b0 + lane < P.requests) from_of(warp)[b0 + lane] = base + v - mine;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
        __syncwarp();
        const int64_t total = base, *start = from_of(warp);
        const int all = parties(total, C);
        const WideShares shares(total, all);
        // the unit and block at or after a place: lane-parallel over the row tiles of its request
        auto find = [&](int64_t at, Unit& u, int& j, int64_t& place) {
            int lo = 0, hi = P.requests - 1;             // the last request that begins at or before `at` (and has rows)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (start[mid] <= at) lo = mid;
                else hi = mid - 1;
            }
            u.b = lo;
            const Request q(P, lo);
            const int tiles = chunk_tiles(q.fresh, P.group, kCtas * kRows), heads = P.cache.kv_heads;
            int64_t from = start[lo];
            for (int r0 = 0; r0 < tiles; r0 += 32) {
                const int64_t each = r0 + lane < tiles ? tile_of(P, q, r0 + lane).blocks + kChunkUnitCost : 0;
                int64_t v = each * heads;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int64_t x = __shfl_up_sync(0xffffffffu, v, s);
                    if (lane >= s) v += x;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, r0 + lane < tiles && from + v > at);
                if (past) {
                    const int who = __ffs((int)past) - 1;
                    const int64_t e = __shfl_sync(0xffffffffu, each, who), end = from + __shfl_sync(0xffffffffu, v, who);
                    const int64_t in = at - (end - e * heads);
                    u.rt = r0 + who;
                    u.head = (int)(in / e);
                    place = end - e * heads + u.head * e;
                    const int k = (int)(at - place);
                    j = k > kChunkUnitCost ? k - kChunkUnitCost : 0;
                    return;
                }
                from += __shfl_sync(0xffffffffu, v, 31);
            }
        };
        const int64_t g0 = c < all ? shares.first(c) : total, g1 = c < all ? shares.first(c + 1) : total;
        Unit u{0, 0, 0};
        int j = 0;
        int64_t place = 0;
        if (g0 < g1) find(warp == 0 ? g0 : g1 - 1, u, j, place);
        if (lane == 0 && warp == 0) {
            out->none = g0 >= g1;
            out->first = u, out->j0 = j, out->place = place;
            *total_out = total;
        } else if (lane == 0) {
            // blocks of the last unit before place g1
            const int64_t k = g1 - place - kChunkUnitCost;
            out->last = u, out->j1 = k > 0 ? (int)k : 0;
        }
    }
    __syncthreads();
    Range r = *out;
    r.none |= r.first.b == r.last.b && r.first.rt == r.last.rt && r.first.head == r.last.head && r.j1 <= r.j0;
    return r;
}

// Whether a tile's keys may have terms S c past the end of binary16's range (all lanes together).
template <int BITS, int D>
__device__ __forceinline__ bool wide_keys(const uint8_t* meta, int lane) {
    constexpr uint32_t kMost = BITS == 4 ? 0x6c00u : 0x5c00u;   // 4096 and 256
    uint2 x = make_uint2(0u, 0u);
    if (8 * lane < KvLayout<BITS, D>::kMeta) x = lds64(meta + 8 * lane);
    const uint32_t over = ((x.x & 0x7fff7fffu) + (0x7fffu - kMost) * 0x10001u) | ((x.y & 0x7fff7fffu) + (0x7fffu - kMost) * 0x10001u);
    return __any_sync(0xffffffffu, (over & 0x80008000u) != 0);
}
// Whether a tile's values S c + Z may, or are no numbers.
template <int BITS, int D>
__device__ __forceinline__ bool wide_values(const uint8_t* meta, int lane) {
    using L = KvLayout<BITS, D>;
    constexpr uint32_t kMostS = BITS == 4 ? 0x6400u : 0x5400u, kMostZ = 0x7400u;   // 1024 and 64, 16384
    uint2 x = make_uint2(0u, 0u);
    if (8 * lane < 2 * L::kMeta) x = lds64(meta + 8 * lane);
    const uint32_t room = (0x7fffu - (8 * lane < L::kMeta ? kMostS : kMostZ)) * 0x10001u;
    const uint32_t over = ((x.x & 0x7fff7fffu) + room) | ((x.y & 0x7fff7fffu) + room);
    return __any_sync(0xffffffffu, (over & 0x80008000u) != 0);
}
// Seldom, and so not in the way of the others' instructions: tiles whose terms are clamped.
template <int BITS, int D, int KEYS>
__device__ __noinline__ void expand_wide_keys(const uint8_t* tile, const uint8_t* meta, uint8_t* stage, uint8_t* zs, int zchunk, int tile_no, int left, int lane) {
    expand_keys<BITS, D, KEYS, true>(tile, meta, stage, zs, zchunk, tile_no, left, lane);
}
template <int BITS, int D, int PARTS>
__device__ __noinline__ void expand_wide_values(const uint8_t* tile, const uint8_t* meta, uint8_t* stage, int tile_no, int left, int lane, int part) {
    expand_values<BITS, D, PARTS, true>(tile, meta, stage, tile_no, left, lane, part);
}

// Value groups of one tile whose S or Z is no number are left out of meta (made 0) and recorded in bad[16], a bit per group
// of the tile's tokens.  Returns whether there is one.  The tile's tokens from .. to - 1, which no row sees, are left out and not recorded:
// theirs may be anything, also numbers whose S c + Z is infinite in binary16, and P = 0 times that is NaN.
template <int BITS, int D>
__device__ __noinline__ bool leave_out_odd_values(uint8_t* meta, uint8_t* bad, int from, int to, int lane) {
    using L = KvLayout<BITS, D>;
    constexpr int G = D / 32;
    uint32_t mask = 0;
    if (lane < 16) {       // lane: the token's place in the rows of S and Z
        // place 4 q + e holds token 2 q + (e & 1) + 8 (e >> 1)
        const int tok = 2 * (lane >> 2) + (lane & 1) + 8 * (lane >> 1 & 1);
        const bool nobodys = tok >= from && tok < to;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint16_t* s = reinterpret_cast<uint16_t*>(meta + g * 32 + 2 * lane);
            uint16_t* z = reinterpret_cast<uint16_t*>(meta + L::kMeta + g * 32 + 2 * lane);
            const bool odd = (*s & 0x7c00u) == 0x7c00u || (*z & 0x7c00u) == 0x7c00u;
            if (odd && !nobodys) mask |= 1u << g;
            if (odd || nobodys) *s = *z = 0;
        }
        bad[tok] = (uint8_t)mask;
    }
    __syncwarp();
    return __any_sync(0xffffffffu, mask != 0);
}

template <int BITS, int D, class T>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams P) {
    using L = KvLayout<BITS, D>;
    using M = ChunkSmem<BITS, D>;
    constexpr int G = D / 32;
    // Binary16 outputs, whose own rounding is no coarser than that of P to binary16: what it left out is multiplied too.
    constexpr bool kFine = IsHalf<T>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // (the swizzle's 1024-byte atoms; alike in both CTAs)
    float* ml = reinterpret_cast<float*>(base + M::kMl);
    float* tops = reinterpret_cast<float*>(base + M::kF);
    __shared__ uint32_t s_tmem;
    __shared__ volatile uint32_t s_there[2][8];        // a block's tiles in the cache, for keys (all of them) and values (no role is 8 ahead of another)
    __shared__ volatile unsigned long long s_odd[kOdd];   // a byte per tile of a block: whether it has values that are no numbers
    __shared__ Range s_range;
    __shared__ int64_t s_total;
    __shared__ int s_last;
    __shared__ volatile int s_past[2][2][4];           // [odd or even blocks]: the last block in which a half's warp met a score past its row's reference
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();

    const uint32_t bars = smem_u32(base + M::kBars);
    // Each CTA's: bytes of keys and values there and used, scores there, O done.  The even CTA's: operands, P and Q there.
    const uint32_t kr_full = bars, kr_empty = kr_full + 8 * M::kRaw, vr_full = kr_empty + 8 * M::kRaw, vr_empty = vr_full + 8 * M::kRaw;
    const uint32_t s_full = vr_empty + 8 * M::kRaw, o_done = s_full + 16, k_full = o_done + 16, v_full = k_full + 16, p_full = v_full + 16;
    const uint32_t q_full = p_full + 16;
    if (tid < 16) s_past[tid >> 3][tid >> 2 & 1][tid & 3] = -1;
    if (tid == 0) {
        for (int i = 0; i < M::kRaw; ++i) {
            mbar_init(kr_full + 8 * i, 1);
            mbar_init(kr_empty + 8 * i, kKeyWarps);
            mbar_init(vr_full + 8 * i, 1);
            mbar_init(vr_empty + 8 * i, kValueWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(s_full + 8 * b, 1);
            mbar_init(o_done + 8 * b, 1);
            mbar_init(k_full + 8 * b, kCtas * kKeyWarps);
            mbar_init(v_full + 8 * b, kCtas * kValueWarps);
            mbar_init(p_full + 8 * b, kCtas * kSoftWarps);
        }
        mbar_init(q_full, kCtas * kSoftWarps);
        fence_mbar_init();
    }
    // (the odd chunks of the Z rows multiply nothing: zero for good)
    for (int i = tid; i < M::kAtom / 16; i += kThreads) sts128(base + M::kZ + 16 * i, 0, 0, 0, 0);
    if (warp == kMmaWarp) tmem_alloc_pair(smem_u32(&s_tmem), kTmemCols);
    fence_async_smem();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_launch_dependents();
    pdl_wait();

    const int c = blockIdx.x / kCtas, C = gridDim.x / kCtas;
    const Range R = range_of(P, c, C, reinterpret_cast<int64_t*>(base + M::kK), &s_total, &s_range);
    int own_abort = 0;
    auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait_bounded<true>(bar, parity & 1u, &own_abort, P.status); };
    auto arrive = [&](uint32_t bar) { mbar_arrive_remote(mapa_shared(bar, 0)); };   // on the even CTA's barrier

    // The softmax warps hold a row's scores, the others little: kThreads * kRegs registers at launch, as many afterwards.
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kLoadWarp || warp == kLoadWarp + 4) {
            // ---------------------------------------------------------------- keys' or values' bytes into their ring
            const int what = warp != kLoadWarp;
            const uint32_t full = what ? vr_full : kr_full, empty = what ? vr_empty : kr_empty;
            const uint32_t dst0 = smem_u32(base + (what ? M::kRawV : M::kRawK));
            const int stage_bytes = what ? M::kRawStageV : M::kRawStageK;
            int s = 0, turn = -1, i = 0;             // blocks
            for (Walk w(P, R); w.more; w.next()) {
                const int32_t* table = P.block_table + w.u.b * P.bt_stride;
                const int end = min(w.t.p1 + 1, w.q.len);
                const uint8_t* src = nullptr;
                for (int j = w.j0; j < w.j1; ++j, ++i) {
                    const int k = j - w.j0;
                    if (k % 4 == 0) {                // addresses of four blocks' tiles, one per lane
                        src = nullptr;
                        if (j + lane / kTiles < w.j1) {
                            const int tile = w.t.block(j + lane / kTiles) * kTiles + lane % kTiles;
                            // (what lies between the sinks and the windows is nobody's, and its pages need not exist)
                            if (tile * kKvTile < end && (tile * kKvTile + kKvTile > w.t.lowest || tile * kKvTile < P.sinks)) {
                                const int pi = tile / P.cache.tiles_per_page, page = table[pi];
                                if (page < 0 || page >= P.cache.num_pages) atomicOr(P.status, kStatusIndex);
                                else
                                    src = P.cache.pages + (((int64_t)page * P.cache.kv_heads + w.u.head) * P.cache.tiles_per_page +
                                                           (tile - pi * P.cache.tiles_per_page)) * (int64_t)L::kBytes;
                            }
                        }
                    }
                    if (turn >= 0) wait(empty + 8 * s, turn);
                    __syncwarp();
                    const uint32_t there = (__ballot_sync(0xffffffffu, src != nullptr) >> (k % 4 * kTiles)) & ((1u << kTiles) - 1u);
                    // (of the keys only this CTA's half is loaded)
                    const uint32_t wanted = what ? there : there & (((1u << M::kTilesHere) - 1u) << (rank * M::kTilesHere));
                    if (lane == 0) {
                        s_there[what][i & 7] = there;
                        if (wanted) mbar_arrive_expect_tx(full + 8 * s, __popc(wanted) * M::kRawTile);
                        else mbar_arrive(full + 8 * s);
                    }
                    __syncwarp();
                    const int no = lane % kTiles;
                    if (lane / kTiles == k % 4 && (wanted >> no & 1u)) {
                        const uint32_t dst = dst0 + s * stage_bytes + (what ? no : no - rank * M::kTilesHere) * M::kRawTile;
                        bulk_load(dst, src + (what ? L::kVc : 0), L::kCodes, full + 8 * s);
                        bulk_load(dst + L::kCodes, src + (what ? L::kVs : L::kKs), 2 * L::kMeta, full + 8 * s);
                    }
                    if (++s == M::kRaw) s = 0, ++turn;
                }
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- all MMAs, one thread of the even CTA
            if (rank == 0) {
                constexpr uint32_t idS = idesc_f16(false, kCtas * kRows, kKeys), idO = idesc_f16(false, kCtas * kRows, D);
                // (descriptors count 16-byte units from their first: a constant each)
                const uint64_t kd = smem_desc_sw128(smem_u32(base + M::kK)), zd = smem_desc_sw128(smem_u32(base + M::kZ));
                const uint64_t vd = smem_desc_sw128(smem_u32(base + M::kV));
                auto scores = [&](int i) {
                    const int b = i & 1;
                    const uint32_t d = tmem + kColS + kKeys * b;
                    const uint64_t k = kd + (b ? M::kKStage / 16 : 0);
                    wait(k_full + 8 * b, i >> 1);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int st = 0; st < D / 16; ++st)
                                tc_mma_f16_ts_pair(d, tmem + kColQ + 8 * st, k + ((part * M::kAtoms + st / 4) * M::kAtom + 32 * (st % 4)) / 16, idS, (part | st) != 0);
                        tc_mma_f16_ts_pair(d, tmem + kColZ, zd + 2 * b, idS, 1);
                        tc_commit_pair(s_full + 8 * b);
                    }
                    __syncwarp();
                };
                int done = 0, u = 0;   // blocks of earlier units, units
                for (Walk w(P, R); w.more; w.next(), ++u) {
                    const int nb = w.j1 - w.j0;
                    wait(q_full, u);
                    tc_fence_after();
                    scores(done);
                    for (int j = 0; j < nb; ++j) {
                        const int i = done + j, b = i & 1;
                        if (j + 1 < nb) scores(i + 1);
                        wait(v_full + 8 * b, i >> 1);
                        wait(p_full + 8 * b, i >> 1);
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t v = vd + (b ? 2 * M::kVAtom / 16 : 0);
#pragma unroll
                            for (int st = 0; st < kKeys / 16; ++st)
                                tc_mma_f16_ts_pair(tmem + kColO, tmem + kColS + kKeys * b + (st / 4) * 64 + 8 * (st % 4), v + ((st / 4) * M::kVAtom + 32 * (st % 4)) / 16,
                                    idO, j != 0 || st != 0);
                            if (kFine) {
#pragma unroll
                                for (int st = 0; st < kKeys / 16; ++st)
                                    tc_mma_f16_ts_pair(tmem + kColO, tmem + kColS + kKeys * b + (st / 4) * 64 + 32 + 8 * (st % 4),
                                        v + ((st / 4) * M::kVAtom + 32 * (st % 4)) / 16, idO, 1);
                            }
                            tc_commit_pair(o_done + 8 * b);
                        }
                        __syncwarp();
                    }
                    done += nb;
                }
            }
            __syncwarp();
        } else if (dq_index(warp) >= 0) {
            // ---------------------------------------------------------------- codes to operands
            const bool keys = dq_index(warp) < kKeyWarps;
            const int wi = keys ? dq_index(warp) : dq_index(warp) - kKeyWarps;
            static_assert(M::kTilesHere == kKeyWarps && kTiles == kValueWarps, "a tile of every block for each warp");
            const uint32_t full = keys ? kr_full : vr_full, empty = keys ? kr_empty : vr_empty;
            uint8_t* raw = base + (keys ? M::kRawK : M::kRawV);
            int s = 0, turn = 0, i = 0;
            for (Walk w(P, R); w.more; w.next()) {
                const int end = min(w.t.p1 + 1, w.q.len);
                for (int j = w.j0; j < w.j1; ++j, ++i) {
                    const int b = i & 1, kb = w.t.block(j);
                    wait(full + 8 * s, turn);
                    // the stage's last MMAs have read it
                    if (keys && i >= 2) wait(s_full + 8 * b, (i >> 1) - 1);
                    if (!keys && i >= 2) wait(o_done + 8 * b, (i >> 1) - 1);
                    const uint32_t there = s_there[keys ? 0 : 1][i & 7];
                    if (keys) {
                        const int no = rank * M::kTilesHere + wi;              // tile of the block
                        const uint8_t* tile = raw + s * M::kRawStageK + wi * M::kRawTile;
                        const int left = there >> no & 1u ? end - kb * kKeys - no * kKvTile : 0;
                        uint8_t *stage = base + M::kK + b * M::kKStage, *zs = base + M::kZ;
                        if (wide_keys<BITS, D>(tile + L::kCodes, lane)) expand_wide_keys<BITS, D, M::kKeysHere>(tile, tile + L::kCodes, stage, zs, 2 * b, wi, left, lane);
                        else expand_keys<BITS, D, M::kKeysHere, false>(tile, tile + L::kCodes, stage, zs, 2 * b, wi, left, lane);
                    } else {
                        uint8_t* tile = raw + s * M::kRawStageV + wi * M::kRawTile;
                        const int left = there >> wi & 1u ? end - kb * kKeys - wi * kKvTile : 0;
                        uint8_t* stage = base + M::kV + (2 * b + wi / 4) * M::kVAtom;
                        bool no_numbers = false;
                        if ((there >> wi & 1u) && wide_values<BITS, D>(tile + L::kCodes, lane)) {
                            const int first = kb * kKeys + wi * kKvTile;
                            no_numbers = leave_out_odd_values<BITS, D>(tile + L::kCodes, base + M::kBad + (i & (kOdd - 1)) * kKeys + wi * kKvTile,
                                                                       P.sinks - first, w.t.lowest - first, lane);
                            expand_wide_values<BITS, D, kCtas>(tile, tile + L::kCodes, stage, wi % 4, left, lane, rank);
                        } else {
                            expand_values<BITS, D, kCtas, false>(tile, tile + L::kCodes, stage, wi % 4, left, lane, rank);
                        }
                        if (lane == 0) reinterpret_cast<volatile uint8_t*>(&s_odd[i & (kOdd - 1)])[wi] = no_numbers;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        arrive((keys ? k_full : v_full) + 8 * b);
                        mbar_arrive(empty + 8 * s);
                    }
                    if (++s == M::kRaw) s = 0, ++turn;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---------------------------------------------------------------- softmax: two threads per row
        const int half = warp >> 2, r = 32 * (warp & 3) + lane;        // keys 64 half .. + 63 of a block, and half of the dimensions
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        // A unit's queries: scaled by a power of two into [2^9, 2^10), their columns in the order of K's rows, and the sums of their
        // groups in two terms; each thread half of its row's dimensions.  Returns what scores are multiplied by.
        auto put_queries = [&](const Row& x) {
            const uint16_t* src = static_cast<const uint16_t*>(P.q) + x.at * P.q_stride + (int64_t)x.qh * D + half * (D / 2);
            uint4 v[D / 16];
#pragma unroll
            for (int k = 0; k < D / 16; ++k) v[k] = x.live ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t y[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(elem_to_float<T>((uint16_t)(y[e >> 1] >> (16 * (e & 1))))));
            }
            tops[half * kRows + r] = top;
            soft_sync();
            top = fmaxf(top, tops[(half ^ 1) * kRows + r]);
            int e = top > 0.f ? 9 - ((int)(__float_as_uint(top) >> 23) - 127) : 0;
            e = min(max(e, -120), 120);
            const float up = pow2i(e);
            __half* z = reinterpret_cast<__half*>(base + M::kGroups) + r * 2 * G;
#pragma unroll
            for (int h = 0; h < G / 2; ++h) {                              // 32 dimensions: 16 columns
                const int g = half * (G / 2) + h;
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 q = v[4 * h + k];
                    const uint32_t y[4] = {q.x, q.y, q.z, q.w};
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = elem_to_float<T>((uint16_t)(y[i >> 1] >> (16 * (i & 1)))) * up;
                    if (BITS == 4) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[4 * k + i] = pack_half2_rn(f[i], f[i + 4]);
                    } else {
                        o[4 * k] = pack_half2_rn(f[0], f[2]), o[4 * k + 1] = pack_half2_rn(f[1], f[3]);
                        o[4 * k + 2] = pack_half2_rn(f[4], f[6]), o[4 * k + 3] = pack_half2_rn(f[5], f[7]);
                    }
                }
                tmem_st16_issue(lanes + kColQ + 16 * g, o);
                float sum = 0.f;                                           // of the rounded values
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 w = unpack2(o[i]);
                    sum += w.x + w.y;
                }
                z[g] = __float2half_rn(sum);
                z[G + g] = __float2half_rn(sum - __half2float(z[g]));
            }
            soft_sync();
            if (half == 0) {
                const uint32_t* y = reinterpret_cast<const uint32_t*>(z);
                tmem_st4_issue(lanes + kColZ, y[0], y[1], G == 4 ? y[2 % G] : 0u, G == 4 ? y[3 % G] : 0u);
                tmem_st4_issue(lanes + kColZ + 4, 0, 0, 0, 0);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(q_full);
            return fmaxf(P.scale_log2 * pow2i(-e), 0x1p-126f);             // (a hidden score is -inf times it)
        };
        int done = 0;
        Walk w(P, R);
        Row row(P, w.q, w.u, rank, r);
        float f = w.more ? put_queries(row) : 0.f;
        while (w.more) {
            const int nb = w.j1 - w.j0, p = row.p;
            float m = -INFINITY, l = 0.f, ref = 0.f;
            uint32_t poison = 0;                                       // groups of dimensions that saw no number
            // the value groups of a block (whose product is done) that this row saw and that are no numbers
            auto odd_values = [&](int i, int kb) {
                if (s_odd[i & (kOdd - 1)] == 0) return;
                for (int k = 0; k < kKeys; ++k) {
                    if (!(reinterpret_cast<volatile uint8_t*>(&s_odd[i & (kOdd - 1)])[k / kKvTile])) continue;
                    const int j = kb * kKeys + k;
                    if (j <= p && (P.window <= 0 || j > p - P.window || j < P.sinks)) poison |= (base + M::kBad)[(i & (kOdd - 1)) * kKeys + k];
                }
            };
            // The product of block i.  A wait tells a barrier's phases apart by their parity alone: the product before on this
            // barrier, of block i - 2, has ended when this is called (see the scores' wait), and the one after waits for P.
            auto wait_o = [&](int i) {
                wait(o_done + 8 * (i & 1), i >> 1);
                tc_fence_after();
            };
            for (int j = 0; j < nb; ++j) {
                const int i = done + j, b = i & 1, kb = w.t.block(w.j0 + j);
                wait(s_full + 8 * b, i >> 1);
                tc_fence_after();
                const uint32_t col = lanes + kColS + kKeys * b + 64 * half;
                const uint32_t there = s_there[0][i & 7] >> (half * kTiles / 2);
                const bool some = !w.t.whole(kb, P.window, P.sinks) || (there & ((1u << kTiles / 2) - 1u)) != (1u << kTiles / 2) - 1u;
                auto hide = [&](int h, uint32_t (&x)[32]) {
                    const int j0 = kb * kKeys + 64 * half + 32 * h;
                    uint32_t sees = below(p + 1 - j0);
                    if (P.window > 0) sees &= ~below(p + 1 - P.window - j0) | below(P.sinks - j0);
                    sees &= (there >> (2 * h) & 1u ? 0xffffu : 0u) | (there >> (2 * h + 1) & 1u ? 0xffff0000u : 0u);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(sees >> k & 1u)) x[k] = 0xff800000u;
                };
                uint32_t xa[32], xb[32];
                auto load = [&] {
                    tmem_ld32_issue(col, xa);
                    tmem_ld32_issue(col + 32, xb);
                    tmem_ld32_wait(xa);
                    tmem_ld32_waited(xb);
                    if (some) hide(0, xa), hide(1, xb);
                };
                float2 sum;
                auto probabilities = [&](uint32_t (&x)[32], uint32_t (&pr)[16], uint32_t (&rest)[16]) {
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), make_float2(f, f), make_float2(-ref, -ref));
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum = add2(sum, e);
                        pr[k / 2] = pack_half2_rn(e.x, e.y);
                        if (kFine) {
                            const float2 h = unpack2(pr[k / 2]);
                            rest[k / 2] = pack_half2_rn(e.x - h.x, e.y - h.y);
                        }
                    }
                };
                uint32_t pa[16], pb[16], ra[16], rb[16];
                bool past = false;
                if (j > 0) {
                    // P by the reference as it is; whether it has to move, in the other half too, turns out meanwhile
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto larger = [&](const uint32_t (&x)[32]) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) top4[k / 2 & 3] = fmaxf(fmaxf(top4[k / 2 & 3], __uint_as_float(x[k])), __uint_as_float(x[k + 1]));
                    };
                    sum = make_float2(0.f, 0.f);
                    load();
                    probabilities(xa, pa, ra);
                    larger(xa);
                    probabilities(xb, pb, rb);
                    larger(xb);
                    past = __any_sync(0xffffffffu, fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * f > m + kPast);
                    if (past && lane == 0) s_past[i & 1][half][warp & 3] = i;
                    rows_sync(warp & 3);
                }
                if (j == 0 || past || s_past[i & 1][half ^ 1][warp & 3] == i) {   // (both warps of the rows alike; in a unit's first block there is no reference yet)
                    load();
                    float mx = -INFINITY, my = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        mx = fmaxf(fmaxf(mx, __uint_as_float(xa[k])), __uint_as_float(xa[k + 1]));
                        my = fmaxf(fmaxf(my, __uint_as_float(xb[k])), __uint_as_float(xb[k + 1]));
                    }
                    mx = fmaxf(mx, my) * f;
                    ml[half * kRows + r] = mx;
                    rows_sync(warp & 3);
                    mx = fmaxf(mx, ml[(half ^ 1) * kRows + r]);
                    const float now = mx > m + kPast ? mx : m, a = m == now ? 1.f : ex2(m - now);
                    if (j > 0 && __any_sync(0xffffffffu, m != now)) {  // each thread its half of O's dimensions
                        wait_o(i - 1);
#pragma unroll 1
                        for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
                            uint32_t o[32];
                            tmem_ld32(lanes + kColO + d, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                            tmem_st32(lanes + kColO + d, o);
                        }
                        load();
                    }
                    l *= a;
                    m = now;
                    ref = now == -INFINITY ? 0.f : now - kPUp;
                    sum = make_float2(0.f, 0.f);
                    probabilities(xa, pa, ra);
                    probabilities(xb, pb, rb);
                }
                tmem_st16_issue(col, pa);      // (over scores that have been read)
                tmem_st16_issue(col + 16, pb);
                if (kFine) {
                    tmem_st16_issue(col + 32, ra);
                    tmem_st16_issue(col + 48, rb);
                }
                l += sum.x + sum.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(p_full + 8 * b);
                // (with a block's scores the product of the block before the last is done too: MMAs end in their order)
                if (j >= 2) odd_values(i - 2, w.t.block(w.j0 + j - 2));
            }

            // ---- the next unit's queries, whose scores are computed while this one's rows are written ----
            const int last = done + nb - 1, kb_last = w.t.block(w.j1 - 1), kb_before = w.t.block(max(w.j1 - 2, w.j0));
            const bool all_here = w.j0 == 0 && w.j1 == w.t.blocks;
            const int64_t place = w.place;
            const int from_first = w.j0, unit_blocks = w.t.blocks;
            const Row here = row;
            float f_next = 0.f;
            w.next();
            if (w.more) {
                row = Row(P, w.q, w.u, rank, r);
                f_next = put_queries(row);
            } else {
                soft_sync();   // (as in there: the maxima's last readers are done)
            }
            // ---- the unit's rows: each thread half of its row's dimensions ----
            ml[half * kRows + r] = l;
            soft_sync();
            l = ml[r] + ml[kRows + r];
            wait_o(last);
            if (nb >= 2) odd_values(last - 1, kb_before);
            odd_values(last, kb_last);
            uint16_t* out = static_cast<uint16_t*>(P.out) + here.at * P.out_stride + (int64_t)here.qh * D;
            auto finish = [&](int d, float (&v)[32], float inv) {      // 32 dimensions from d on
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    alignas(16) T y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = (T)(v[k + e] * inv);
                    *reinterpret_cast<uint4*>(out + d + k) = *reinterpret_cast<const uint4*>(y);
                }
            };
            auto finish_sum = [&](float top, float total) {
                if (half == 0 && here.live && P.lse)
                    P.lse[here.at * P.q_heads + here.qh] = total == 0.f ? -INFINITY : (top + log2f(total) - kPUp) * 0.6931471805599453f;
            };
            constexpr int kSlot = kRows * (D + 2);
            float* slot = P.part + (int64_t)((2 * c + (from_first == 0 ? 1 : 0)) * kCtas + rank) * kSlot;   // [D / 4][rows] of four, then [rows] m, l
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
                float v[32];
                tmem_ld32(lanes + kColO + d, reinterpret_cast<uint32_t(&)[32]>(v));
                if (poison >> (d / 32) & 1u) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = NAN;
                }
                if (all_here) {
                    if (here.live) finish(d, v, inv);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<float4*>(slot + ((d + k) / 4 * kRows + r) * 4) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                }
            }
            if (all_here) {
                finish_sum(m, l);
            } else {
                if (half == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(m, l);
                const WideShares shares(s_total, parties(s_total, C));
                const int64_t from = place + kChunkUnitCost;
                const int c0 = shares.of(from), c1 = shares.of(from + unit_blocks - 1);
                soft_sync();
                // (release of what the block wrote before the barrier, acquire of what the others did)
                if (tid == 0) s_last = arrive_gpu(P.counters + c0 * kCtas + rank) == (unsigned)(c1 - c0);
                soft_sync();
                if (s_last) {
                    auto part = [&](int k) { return P.part + (int64_t)((2 * (c0 + k) + (k == 0 ? 1 : 0)) * kCtas + rank) * kSlot; };
                    auto sums = [&](int k) { return __ldcg(reinterpret_cast<const float2*>(part(k) + kRows * D + 2 * r)); };
                    float top = -INFINITY, total = 0.f;
                    for (int k = 0; k <= c1 - c0; ++k) top = fmaxf(top, sums(k).x);
                    const float mine = top == -INFINITY ? 0.f : top;
                    for (int k = 0; k <= c1 - c0; ++k) total += sums(k).y * ex2(sums(k).x - mine);
                    const float all = total == 0.f ? 0.f : 1.f / total;
#pragma unroll 1
                    for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
                        float v[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0.f;
#pragma unroll 1
                        for (int k = 0; k <= c1 - c0; ++k) {
                            const float e = ex2(sums(k).x - mine);
                            const float* o = part(k);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float4 x = __ldcg(reinterpret_cast<const float4*>(o + ((d / 4 + q) * kRows + r) * 4));
                                v[4 * q] = fmaf(x.x, e, v[4 * q]), v[4 * q + 1] = fmaf(x.y, e, v[4 * q + 1]);
                                v[4 * q + 2] = fmaf(x.z, e, v[4 * q + 2]), v[4 * q + 3] = fmaf(x.w, e, v[4 * q + 3]);
                            }
                        }
                        if (here.live) finish(d, v, all);
                    }
                    finish_sum(top, total);
                    if (tid == 0) P.counters[c0 * kCtas + rank] = 0;
                }
            }
            tc_fence_before();
            soft_sync();   // both halves are done with O and the sums
            done += nb;
            f = f_next;
        }
    }
    tc_fence_before();
    cluster_sync_all();   // (no arrival or tensor-memory access of either CTA is still to come)
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// Clusters of the kernel that fit on the device at once (0 on error); sets its shared-memory attribute.  Kept per device.
template <int BITS, int D, class T>
int pairs_at_once(int device, int max_smem) {
    static std::mutex mu;
    static int known[kMaxDevices] = {};
    constexpr int smem = ChunkSmem<BITS, D>::kSize;
    if (device < 0 || device >= kMaxDevices || smem > max_smem) return 0;
    const std::lock_guard<std::mutex> lock(mu);
    if (known[device] == 0) {
        auto kernel = chunk_kernel<BITS, D, T>;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
        cudaGetLastError();
        known[device] = n;
    }
    return known[device];
}

template <int BITS, int D, class T>
lq_status run(lq_handle h, const ChunkParams& P, cudaStream_t stream) {
    const int pairs = pairs_at_once<BITS, D, T>(h->device, h->max_smem_optin);
    if (pairs < 1) return LQ_ERR_UNSUPPORTED;
    if ((size_t)pairs * 2 > h->num_counters || (size_t)pairs * 4 * kRows * (D + 2) > h->partial_floats) return LQ_ERR_WORKSPACE;
    return launch_overlapped(chunk_kernel<BITS, D, T>, dim3(2 * pairs), kThreads, ChunkSmem<BITS, D>::kSize, stream, P);
}

}  // namespace

lq_status launch_kv_chunk(lq_handle h, const lq_kv_cache& c, const lq_kv_chunk_args& a, cudaStream_t stream) {
    ChunkParams P = {};
    P.cache = KvView{static_cast<uint8_t*>(c.pages), c.num_pages, c.page_size, c.kv_heads, c.page_size / kKvTile};
    P.q = a.q, P.out = a.out, P.lse = a.lse;
    P.q_stride = a.q_token_stride, P.out_stride = a.out_token_stride, P.bt_stride = a.block_table_stride;
    P.block_table = a.block_table, P.lens = a.lens, P.starts = a.starts;
    P.requests = a.batch, P.tokens = a.tokens, P.group = a.q_heads / c.kv_heads, P.q_heads = a.q_heads;
    P.max_len = a.max_pages * c.page_size;
    P.window = a.window, P.sinks = a.sinks;
    P.scale_log2 = a.scale * 1.4426950408889634f;
    P.part = h->partials, P.counters = h->counters, P.status = h->status_flag;
    const bool bf16 = a.dtype == LQ_BF16;
    if (c.head_dim == 128) {
        if (c.bits == 4) return bf16 ? run<4, 128, __nv_bfloat16>(h, P, stream) : run<4, 128, __half>(h, P, stream);
        return bf16 ? run<8, 128, __nv_bfloat16>(h, P, stream) : run<8, 128, __half>(h, P, stream);
    }
    if (c.bits == 4) return bf16 ? run<4, 64, __nv_bfloat16>(h, P, stream) : run<4, 64, __half>(h, P, stream);
    return bf16 ? run<8, 64, __nv_bfloat16>(h, P, stream) : run<8, 64, __half>(h, P, stream);
}

}  // namespace lq
