// Log probabilities of given tokens, entropy and the top alternatives of rows of logits, and their gradient.
//
//   s = sum_i e^(x_i - m),  w = sum_i e^(x_i - m) (x_i - m),  m = max_i x_i
//   lse = m + ln s,  logprob = x_t - m - ln s,  entropy = ln s - w / s
//   d x_i = p_i (-g - h (ln p_i + entropy)) + g [i = t],  p_i = e^(x_i - lse), g and h the gradients that came
//
// One fp32 lse is off by up to 2^-24 of its size, which would go whole into every p_i (logits about 1e5: 0.2 %; a row of the type's
// lowest value: p = 1 for each).  So the forward pass leaves what its rounding dropped as well, and ln p_i = d - rest with d = x_i - lse,
// which is exact wherever the rest matters; |rest| <= ln s, as m is an fp32 number.  The rest goes into the sums that are formed anyway.
//
// Bound by the logits' bytes: one pass forward, one more (and the gradient written) backward.  A thread keeps its own
// running m, s and w over vectors of 16 bytes, four in flight, so that nothing passes between threads before a row's end; five
// blocks share an SM, so that some load while others add.  A block takes a row, or one of a row's equal parts, as many as make the
// device's last turn of blocks a full one.  The last block to arrive joins a row's parts in their order (results repeat bit for bit).
//
// The best k of a row: the k-th largest of the threads' own maxima bounds the k-th largest logit from below, and few
// threads hold anything above it.  Their chunks that do are read once more (from L2) and what passes the bound goes
// to shared memory, where it is ranked by counting.  A logit and its index make one 64-bit key, larger for the larger logit
// and then for the lower index, so no two are equal and no order of arrival matters.
//
// Measured: 2048 rows of 32000 bf16 logits 25.1 us (5.2 TB/s of a copy's 6.8), 1024 of 131072 47 us (5.7); the gradient of those
// 82 to 84 us (6.4 to 6.5 TB/s); 333 rows of 50021 fp32 logits with 20 alternatives 22.5 us (3.0); one row of 32000 with 5 alternatives 7.6,
// latency (a launch, the pass, the alternatives, the joining of parts).  On the way: packed pairs and maxima of words instead of
// values one by one 38 -> 25; alternatives bounded by the threads' maxima instead of a search by bits over all values 63 -> 23.
// Not kept: one block per place, taking parts in turn with the next one's loads under way (2048 x 32000: 34).

#include <algorithm>

#include "lq_internal.h"
#include "lq_tma.cuh"
#include "lq_common.cuh"

namespace lq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPerSm = 5;                    // blocks that share an SM (four with alternatives)
constexpr int kVecs = 4;                     // 16-byte loads of a chunk, per thread
constexpr int kMaxSplits = 32;               // parts of a row (a warp joins them)
constexpr int kKept = 16;                    // chunks whose largest values are kept apart (a power of two)
static_assert(kThreads == 256 && kVecs == 4, "items: eight bits of a thread, four lanes of a chunk");
constexpr int kSpare = 16;                   // threads that may pass the bound of the best k besides k of them
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -150.f;               // e^kFar is 0: what infinitely improbable logits are held at

struct LogprobParams {
    const void* x;
    int64_t stride;
    const int64_t* tokens;
    float *logprob, *entropy, *lse, *rest;
    int64_t* top_ids;
    float* top_logprobs;
    int n, V, top, splits;
    float* part;                             // [row][split]: m, s, w
    unsigned long long* keys;                // [row][split][top]
    unsigned* counters;                      // one per row, zero between calls
    int* status;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ unsigned arrive(unsigned* count) {
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
    return old;
}

template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return reinterpret_cast<float2&>(d);
}

// The words of 16 bytes of values: pairs as fp32, the larger of two words' values one by one (a NaN loses), and 16 bytes of
// which values that do not exist are -inf.
template <class T>
struct Words;
template <>
struct Words<float> {
    static constexpr int kPairs = 2;         // pairs of values in 16 bytes
    static constexpr int kLow = 0;           // low bits of an ordered value that say nothing: all 0, or all 1 below the order of 0
    __device__ __forceinline__ static float2 pair(const uint4& v, int i) {
        return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y)) : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) { return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))); }
    __device__ __forceinline__ static float largest(uint32_t a) { return __uint_as_float(a); }
    __device__ __forceinline__ static void put(uint32_t (&w)[4], int i, float v) { w[i] = __float_as_uint(v); }
    static constexpr uint32_t kNone = 0xff800000u;
};
template <>
struct Words<__half> {
    static constexpr int kPairs = 4, kLow = 13;
    __device__ __forceinline__ static float2 pair(const uint4& v, int i) {
        const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        return __half22float2(reinterpret_cast<const __half2&>(w));
    }
    __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ __forceinline__ static float largest(uint32_t a) { return fmaxf(half_bits_to_float((uint16_t)a), half_bits_to_float((uint16_t)(a >> 16))); }
    __device__ __forceinline__ static void put(uint32_t (&w)[4], int i, __half v) {
        w[i >> 1] = (w[i >> 1] & (i & 1 ? 0xffffu : 0xffff0000u)) | (uint32_t)__half_as_ushort(v) << (16 * (i & 1));
    }
    static constexpr uint32_t kNone = 0xfc00fc00u;
};
template <>
struct Words<__nv_bfloat16> {
    static constexpr int kPairs = 4, kLow = 16;
    __device__ __forceinline__ static float2 pair(const uint4& v, int i) {
        const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ __forceinline__ static float largest(uint32_t a) { return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)); }
    __device__ __forceinline__ static void put(uint32_t (&w)[4], int i, __nv_bfloat16 v) {
        w[i >> 1] = (w[i >> 1] & (i & 1 ? 0xffffu : 0xffff0000u)) | (uint32_t)__bfloat16_as_ushort(v) << (16 * (i & 1));
    }
    static constexpr uint32_t kNone = 0xff80ff80u;
};

// The aligned 16 bytes of values a .. of a row of V values (a may be negative); -inf outside the row.  Only those at a
// row's ends are read value by value, so nothing outside the row is touched.
template <class T>
__device__ __forceinline__ uint4 load_words(const T* row, int64_t a, int V) {
    constexpr int VEC = 16 / sizeof(T);
    if (a >= 0 && a <= V - VEC) return *reinterpret_cast<const uint4*>(row + a);
    uint32_t w[4] = {Words<T>::kNone, Words<T>::kNone, Words<T>::kNone, Words<T>::kNone};
    if (a < V) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (a + i >= 0 && a + i < V) Words<T>::put(w, i, row[a + i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Orders like the values (NaN above all, -0 as 0); never 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = x != x ? 0x7fc00000u : __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }

struct Sums {
    float m, s, w;
    // about the maximum `to` instead of m (to >= m)
    __device__ __forceinline__ void move(float to) {
        const float d = max_nan(m - (to == -INFINITY ? 0.f : to), kFar), e = ex2f(d * kLog2e);
        w = (w + s * d) * e;
        s *= e;
        m = to;
    }
    // with the other lanes' (the same in all of them)
    __device__ __forceinline__ void join_lanes() {
        float top = m;
#pragma unroll
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        move(top);
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, k);
            w += __shfl_xor_sync(0xffffffffu, w, k);
        }
    }
};

// A block's part of a row: values from a 16-byte boundary on, in chunks of kVecs runs of 16 bytes per thread.
template <class T>
struct Part {
    static constexpr int VEC = 16 / sizeof(T), kRun = kThreads * VEC, kChunk = kVecs * kRun;
    const T* x;
    int row, split, before, c0, c1;
    __device__ __forceinline__ Part(const LogprobParams& P, int unit) {
        row = (unsigned)unit / (unsigned)P.splits, split = unit - row * P.splits;
        x = static_cast<const T*>(P.x) + row * P.stride;
        before = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        const unsigned chunks = ((unsigned)P.V + before + kChunk - 1) / kChunk;      // (below 2^20)
        c0 = (int)(chunks * split / (unsigned)P.splits), c1 = (int)(chunks * (split + 1) / (unsigned)P.splits);
    }
    // the first value of a thread's run u of a chunk
    __device__ __forceinline__ int at(int chunk, int u, int thread) const { return chunk * kChunk + u * kRun + thread * VEC - before; }
    __device__ __forceinline__ int at(int chunk, int u) const { return at(chunk, u, threadIdx.x); }
    __device__ __forceinline__ void load(int chunk, int V, uint4 (&v)[kVecs]) const {
        const int a = at(chunk, 0);
        if (chunk * kChunk >= before && (chunk + 1) * kChunk - before <= V) {        // (the block together)
            const uint4* p = reinterpret_cast<const uint4*>(x + a);
#pragma unroll
            for (int u = 0; u < kVecs; ++u) v[u] = p[u * kThreads];
        } else {
#pragma unroll
            for (int u = 0; u < kVecs; ++u) v[u] = load_words<T>(x, a + u * kRun, V);
        }
    }
};

template <class T>
__device__ __forceinline__ uint32_t largest_word(const uint4& v) {
    return Words<T>::larger(Words<T>::larger(v.x, v.y), Words<T>::larger(v.z, v.w));
}

template <int TOP>
struct Shared {
    static constexpr int kRoom = TOP ? kMaxSplits * TOP > 1024 ? kMaxSplits * TOP : 1024 : 1;   // candidates at a time
    unsigned long long found[kRoom], best[TOP ? TOP : 1];
    float big[TOP ? kKept : 1][kThreads];                       // each thread's largest value in every kKept-th chunk
    Sums sums[kWarps];
    uint32_t largest[TOP ? kThreads : 1], bound;
    uint16_t item[TOP ? kKept * kThreads : 1];                  // thread, kept chunk in bits 8 .., and whether it may hold a NaN
    int pass, count, items, last;
};

// The `top` largest of the first n keys of found[] to best[], largest first (0 where there are fewer).  All threads call it.
template <int TOP>
__device__ __forceinline__ void rank_keys(Shared<TOP>& S, int n, int top) {
    __syncthreads();
    for (int i = threadIdx.x; i < top; i += kThreads) S.best[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long mine = S.found[i];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) above += S.found[j] > mine;
        if (mine && above < top) S.best[above] = mine;
    }
    __syncthreads();
}

// Calls f with the keys of this thread's values that may reach the bound.  Chunks and vectors that stay below it are passed
// over by their largest value, unless they may hold a NaN, which no maximum shows.
template <class T, int TOP, class F>
__device__ __forceinline__ void each_key(const Shared<TOP>& S, const Part<T>& part, int V, uint32_t bound, bool any_nan, F&& f) {
    for (int c = part.c0; c < part.c1; ++c) {
        if (!any_nan && ordered(S.big[(c - part.c0) % kKept][threadIdx.x]) < bound) continue;
        uint4 v[kVecs];
        part.load(c, V, v);
#pragma unroll 1
        for (int u = 0; u < kVecs; ++u) {
            const uint4 x = u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3];
            if (!any_nan && ordered(Words<T>::largest(largest_word<T>(x))) < bound) continue;
            const int j = part.at(c, u);
#pragma unroll 1
            for (int i = 0; i < Words<T>::kPairs; ++i) {
                const float2 p = Words<T>::pair(x, i);
                if (j + 2 * i >= 0 && j + 2 * i < V) f(ordered(p.x), (uint32_t)(j + 2 * i));
                if (j + 2 * i + 1 >= 0 && j + 2 * i + 1 < V) f(ordered(p.y), (uint32_t)(j + 2 * i + 1));
            }
        }
    }
}

// The part's `top` largest keys to S.best.  m: this thread's largest value (numbers only), any_nan: whether it may have met a NaN.
template <class T, int TOP>
__device__ __noinline__ void find_top(Shared<TOP>& S, const Part<T>& part, int V, int top, float m, bool any_nan) {
    const int tid = threadIdx.x;
    uint32_t o = part.at(part.c0, 0) < V ? ordered(m) : 0u;              // (its first run is the one that begins first)
    if (any_nan) each_key<T>(S, part, V, 0u, true, [&](uint32_t k, uint32_t) { o = max(o, k); });
    // t: a bound that `top` threads pass, and few more where their largest values differ: the bits of the top-th largest,
    // found one by one below those that all have in common
    unsigned long long least = 1;                                       // a key has to be this large
    S.largest[tid] = o;
    __syncthreads();
    if (tid < 32) {                                                     // (one warp: a round of the block's barriers takes twice as long)
        uint32_t all[kWarps], t = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) all[k] = S.largest[32 * k + tid];
        auto passing = [&](uint32_t bound) {
            int n = 0;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) n += all[k] >= bound;
            return __reduce_add_sync(0xffffffffu, n);
        };
        int pass = passing(1u);
        for (int b = 31; b >= Words<T>::kLow && pass > top + kSpare; --b) {
            const int n = passing(t | 1u << b);
            if (n >= top) t |= 1u << b, pass = n;
        }
        if (tid == 0) S.bound = t, S.pass = pass;
    }
    __syncthreads();
    uint32_t t = S.bound;
    const int pass = S.pass;
    if (t != 0) {            // (0: few threads have values at all)
        uint32_t cut = 0xffffffffu;
        if (pass > top + kSpare) {
            // many equal ones: of the threads whose largest is t, those with the lowest index of one
            if (!(t >> 31)) t |= (1u << Words<T>::kLow) - 1u;
            const int above = __syncthreads_count(o > t);
            uint32_t first = 0xffffffffu;
            if (o == t) each_key<T>(S, part, V, t, any_nan, [&](uint32_t k, uint32_t j) { first = k == t && j < first ? j : first; });
            cut = 0;
            for (int b = 30; b >= 0; --b) {                             // the largest index with fewer than top - above below it
                const uint32_t up = cut | 1u << b;
                if (__syncthreads_count(first < up) < top - above) cut = up;
            }
        }
        least = (unsigned long long)t << 32 | (0xffffffffu - cut);
    }
    for (;;) {
        const uint32_t bound = (uint32_t)(least >> 32);
        if (tid == 0) S.count = S.items = 0;
        __syncthreads();
        // threads' chunks that may reach the bound, then four lanes for each of them: one wait for L2 however many there are
        const int kept = min(kKept, part.c1 - part.c0);
        for (int k = 0; k < kept; ++k)
            if (any_nan || (o != 0 && ordered(S.big[k][tid]) >= bound))
                S.item[atomicAdd(&S.items, 1)] = (uint16_t)(tid | k << 8 | (any_nan ? 0x8000 : 0));
        __syncthreads();
        for (int i = tid >> 2; i < S.items; i += kThreads / 4) {
            const int item = S.item[i];
            for (int c = part.c0 + (item >> 8 & (kKept - 1)); c < part.c1; c += kKept) {
                const int j = part.at(c, tid & 3, item & 255);
                const uint4 x = load_words<T>(part.x, j, V);
                if (!(item & 0x8000) && ordered(Words<T>::largest(largest_word<T>(x))) < bound) continue;
#pragma unroll
                for (int e = 0; e < 2 * Words<T>::kPairs; ++e) {
                    const float2 p = Words<T>::pair(x, e / 2);
                    const unsigned long long key = (unsigned long long)ordered(e & 1 ? p.y : p.x) << 32 | (0xffffffffu - (uint32_t)(j + e));
                    if (j + e >= 0 && j + e < V && key >= least) {
                        const int at = atomicAdd(&S.count, 1);
                        if (at < Shared<TOP>::kRoom) S.found[at] = key;
                    }
                }
            }
        }
        __syncthreads();
        const int n = S.count;
        rank_keys(S, min(n, Shared<TOP>::kRoom), top);
        if (n <= Shared<TOP>::kRoom) return;
        least = S.best[top - 1];             // more than there is room for: what was found raises the bound
        __syncthreads();
    }
}

// TOP: the largest k this variant has room for, 0: no alternatives.
template <class T, int TOP>
__global__ void __launch_bounds__(kThreads, TOP ? kPerSm - 1 : kPerSm) logprobs_kernel(const __grid_constant__ LogprobParams P) {
    __shared__ Shared<TOP> S;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = P.V, top = P.top;
    const Part<T> part(P, blockIdx.x);
    Sums mine{-INFINITY, 0.f, 0.f};
    for (int c = part.c0; c < part.c1; ++c) {
        uint4 v[kVecs];
        part.load(c, V, v);
        uint32_t big = largest_word<T>(v[0]);
#pragma unroll
        for (int u = 1; u < kVecs; ++u) big = Words<T>::larger(big, largest_word<T>(v[u]));
        const float top_here = Words<T>::largest(big), m = fmaxf(mine.m, top_here);
        if (TOP) {
            float* b = &S.big[(c - part.c0) % kKept][tid];
            *b = c - part.c0 < kKept ? top_here : fmaxf(*b, top_here);
        }
        if (m != mine.m) mine.move(m);
        const float ref = m == -INFINITY ? 0.f : m;
        float2 s = make_float2(0.f, 0.f), w = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int i = 0; i < Words<T>::kPairs; ++i) {
                float2 d = add2(Words<T>::pair(v[u], i), make_float2(-ref, -ref));
                d = make_float2(max_nan(d.x, kFar), max_nan(d.y, kFar));
                const float2 y = mul2(d, make_float2(kLog2e, kLog2e)), e = make_float2(ex2f(y.x), ex2f(y.y));
                s = add2(s, e);
                w = fma2(e, d, w);
            }
        mine.s += s.x + s.y;
        mine.w += w.x + w.y;
    }
    const float own = mine.m;
    const bool any_nan = mine.s != mine.s;
    mine.join_lanes();
    if (lane == 0) S.sums[warp] = mine;
    __syncthreads();
    const int64_t slot = (int64_t)part.row * P.splits + part.split;
    if (TOP) {
        find_top<T, TOP>(S, part, V, top, own, any_nan);
        if (P.splits > 1) {
            for (int i = tid; i < top; i += kThreads) P.keys[slot * top + i] = S.best[i];
            __syncthreads();
        }
    } else if (warp != 0) {
        return;
    }
    // ---- the block's sums, then the row's (one warp; with alternatives all of them, alike) ----
    Sums all = lane < kWarps ? S.sums[lane] : Sums{-INFINITY, 0.f, 0.f};
    all.join_lanes();
    if (P.splits > 1) {
        bool last = false;
        if (tid == 0) {
            float* p = P.part + 3 * slot;
            p[0] = all.m, p[1] = all.s, p[2] = all.w;
            last = arrive(P.counters + part.row) == (unsigned)(P.splits - 1);
            if (last) P.counters[part.row] = 0;
        }
        if (TOP) {
            if (tid == 0) S.last = last;
            __syncthreads();
            last = S.last;
            __syncthreads();
        } else {
            last = __shfl_sync(0xffffffffu, last, 0);
            __syncwarp();        // (the other lanes read the parts behind lane 0's acquisition: a shuffle alone orders no memory)
        }
        if (!last) return;
        const float* p = P.part + 3 * ((int64_t)part.row * P.splits + lane);
        all = lane < P.splits ? Sums{__ldcg(p), __ldcg(p + 1), __ldcg(p + 2)} : Sums{-INFINITY, 0.f, 0.f};
        all.join_lanes();
        if (TOP) {
            // the parts' last keys bound the row's from below
            const int n = P.splits * top;
            const unsigned long long* keys = P.keys + (int64_t)part.row * n;
            unsigned long long bound = lane < P.splits ? __ldcg(keys + lane * top + top - 1) : 0;
#pragma unroll
            for (int k = 16; k; k >>= 1) bound = max(bound, __shfl_xor_sync(0xffffffffu, bound, k));
            if (tid == 0) S.count = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const unsigned long long key = __ldcg(keys + i);
                if (key && key >= bound) S.found[atomicAdd(&S.count, 1)] = key;
            }
            __syncthreads();
            rank_keys(S, S.count, top);
        }
    }
    const float ref = all.m == -INFINITY ? 0.f : all.m, ln = logf(all.s);
    const bool none = all.s == 0.f;      // no token is possible
    if (TOP) {
        for (int i = tid; i < top; i += kThreads) {
            const unsigned long long k = S.best[i];
            P.top_ids[(int64_t)part.row * top + i] = (int64_t)(0xffffffffu - (uint32_t)k);
            P.top_logprobs[(int64_t)part.row * top + i] = none ? -INFINITY : unordered((uint32_t)(k >> 32)) - ref - ln;
        }
    }
    if (tid == 0) {
        if (P.entropy) P.entropy[part.row] = none ? 0.f : ln - all.w / all.s;
        const float lse = __fadd_rn(ref, ln);
        if (P.lse) P.lse[part.row] = none ? -INFINITY : lse;
        if (P.rest) {                    // ref + ln - lse, exactly (whichever of the two is the larger)
            const float of_ln = __fsub_rn(lse, ref);
            P.rest[part.row] = none ? 0.f : __fadd_rn(__fsub_rn(ref, __fsub_rn(lse, of_ln)), __fsub_rn(ln, of_ln));
        }
        const int64_t t = P.tokens[part.row];
        if (t >= V) atomicOr(P.status, kStatusIndex);
        P.logprob[part.row] = t < 0 || t >= V ? 0.f : none ? -INFINITY : to_float(part.x[t]) - ref - ln;
    }
}

struct GradParams {
    const void* x;
    int64_t stride;
    void* dx;
    int64_t dx_stride;
    const int64_t* tokens;
    const float *lse, *rest, *entropy, *d_logprob, *d_entropy;
    int n, V, splits;
};

// Blocks of a row take its vectors in turn.  (Five to an SM: left to itself the compiler takes fewer registers, and 1024 rows of 131072
// bf16 logits 87 us, not 84.)
template <class T>
__global__ void __launch_bounds__(kThreads, kPerSm) logprobs_grad_kernel(const __grid_constant__ GradParams P) {
    constexpr int VEC = 16 / sizeof(T);
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x / P.splits, split = blockIdx.x - row * P.splits, V = P.V;
    const T* x = static_cast<const T*>(P.x) + row * P.stride;
    T* dx = static_cast<T*>(P.dx) + row * P.dx_stride;
    const int before = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    // vectors are written whole where the two rows lie alike
    const bool alike = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
    const int64_t t = P.tokens[row];
    const bool given = t >= 0 && t < V;
    const float lse = P.lse[row], ref = lse == -INFINITY ? 0.f : lse, rest = P.rest ? P.rest[row] : 0.f;
    const float g = given && P.d_logprob ? P.d_logprob[row] : 0.f;
    const float h = P.d_entropy ? P.d_entropy[row] : 0.f, H = h != 0.f ? P.entropy[row] : 0.f;
    const float c = -g - h * (H - rest), far = -rest * kLog2e;
    auto gradient = [&](float2 v) {
        float2 d = add2(v, make_float2(-ref, -ref));
        d = make_float2(max_nan(d.x, kFar), max_nan(d.y, kFar));
        const float2 y = fma2(d, make_float2(kLog2e, kLog2e), make_float2(far, far)), p = make_float2(ex2f(y.x), ex2f(y.y));
        return mul2(p, fma2(d, make_float2(-h, -h), make_float2(c, c)));
    };
    const int64_t step = (int64_t)P.splits * kThreads * VEC;
    for (int64_t a0 = ((int64_t)split * kThreads + threadIdx.x) * VEC - before; a0 < V; a0 += kVecs * step) {
        uint4 v[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) v[u] = load_words<T>(x, a0 + u * step, V);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int64_t a = a0 + u * step;
            alignas(16) T y[VEC];
#pragma unroll
            for (int i = 0; i < Words<T>::kPairs; ++i) {
                const float2 r = gradient(Words<T>::pair(v[u], i));
                y[2 * i] = (T)r.x, y[2 * i + 1] = (T)r.y;
            }
            if (alike && a >= 0 && a + VEC <= V) *reinterpret_cast<uint4*>(dx + a) = *reinterpret_cast<const uint4*>(y);
            else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (a + i >= 0 && a + i < V) dx[a + i] = y[i];
            }
            if (given && t >= a && t < a + VEC) {    // (the token's own, over what this thread has just written)
#pragma unroll
                for (int i = 0; i < Words<T>::kPairs; ++i) {
                    const float2 f = Words<T>::pair(v[u], i), r = gradient(f);
                    if (a + 2 * i == t) dx[t] = (T)(r.x + g);
                    if (a + 2 * i + 1 == t) dx[t] = (T)(r.y + g);
                }
            }
        }
    }
}

template <class T, int TOP>
lq_status run(const LogprobParams& P, cudaStream_t stream) {
    return launch_overlapped(logprobs_kernel<T, TOP>, dim3((unsigned)P.n * P.splits), kThreads, 0, stream, P);
}

template <class T>
lq_status run_top(const LogprobParams& P, cudaStream_t stream) {
    if (P.top == 0) return run<T, 0>(P, stream);
    return P.top <= 32 ? run<T, 32>(P, stream) : run<T, kMaxLogprobTop>(P, stream);
}

}  // namespace

lq_status launch_logprobs(lq_handle h, const lq_logprobs_args& a, cudaStream_t stream) {
    LogprobParams P = {};
    P.x = a.logits, P.stride = a.row_stride, P.tokens = a.tokens;
    P.logprob = a.logprob, P.entropy = a.entropy, P.lse = a.lse, P.rest = a.lse_rest, P.top_ids = a.top_ids, P.top_logprobs = a.top_logprobs;
    P.n = a.n, P.V = a.vocab, P.top = a.top;
    P.status = h->status_flag;
    // Parts of a row.  In units of the time in which all resident blocks read a chunk each (1.5 us): the bytes, or a block's
    // own chunks one after another (0.4 each), and what a turn of the blocks costs besides: 1, where parts are joined 1 more,
    // where alternatives are sought 2.5 more.
    const int64_t chunk = kThreads * kVecs * 16 / (a.dtype == LQ_F32 ? 4 : 2), chunks = (a.vocab + chunk - 1) / chunk;
    const int64_t slots = (int64_t)(a.top ? kPerSm - 1 : kPerSm) * h->num_sms;
    int splits = 1;
    double least = 0.0;
    for (int s = 1; s <= std::min<int64_t>(chunks, kMaxSplits); ++s) {
        const int64_t units = (int64_t)a.n * s, turns = (units + slots - 1) / slots;
        if (s > 1 && ((size_t)a.n > h->num_counters || (size_t)units * (a.top * 8 + 12) > h->partial_floats * sizeof(float) || units > 0x7fffffff))
            break;
        const double read = std::max((double)a.n * chunks / slots, 0.4 * turns * ((chunks + s - 1) / s));
        const double cost = read + turns * (1.0 + (s > 1 ? 1.0 : 0.0) + (a.top ? 2.5 : 0.0));
        if (s == 1 || cost < least) least = cost, splits = s;
    }
    P.splits = splits;
    P.keys = reinterpret_cast<unsigned long long*>(h->partials);
    P.part = h->partials + (size_t)a.n * splits * a.top * 2;
    P.counters = h->counters;
    if (a.dtype == LQ_F32) return run_top<float>(P, stream);
    return a.dtype == LQ_F16 ? run_top<__half>(P, stream) : run_top<__nv_bfloat16>(P, stream);
}

lq_status launch_logprobs_grad(lq_handle h, const lq_logprobs_grad_args& a, cudaStream_t stream) {
    GradParams P = {};
    P.x = a.logits, P.stride = a.row_stride, P.dx = a.d_logits, P.dx_stride = a.d_row_stride, P.tokens = a.tokens;
    P.lse = a.lse, P.rest = a.lse_rest, P.entropy = a.entropy, P.d_logprob = a.d_logprob, P.d_entropy = a.d_entropy;
    P.n = a.n, P.V = a.vocab;
    const int e = a.dtype == LQ_F32 ? 4 : 2, chunk = kThreads * kVecs * 16 / e;
    const int64_t want = std::max<int64_t>(1, (int64_t)h->num_sms * 16 / a.n);
    P.splits = (int)std::min<int64_t>(want, ((int64_t)a.vocab + chunk - 1) / chunk);
    const dim3 grid((unsigned)a.n * P.splits);
    if (a.dtype == LQ_F32) return launch_overlapped(logprobs_grad_kernel<float>, grid, kThreads, 0, stream, P);
    return a.dtype == LQ_F16 ? launch_overlapped(logprobs_grad_kernel<__half>, grid, kThreads, 0, stream, P)
                             : launch_overlapped(logprobs_grad_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, P);
}

}  // namespace lq
