// Log probabilities of given tokens, entropy and the top alternatives of rows of logits, and their gradient.
//
//   s = sum_i e^(x_i - m),  w = sum_i e^(x_i - m) (x_i - m),  m = max_i x_i
//   lse = m + ln s,  logprob = x_t - m - ln s,  entropy = ln s - w / s
//   d x_i = p_i (-g - h (ln p_i + entropy)) + g [i = t],  p_i = e^(x_i - lse), g and h the gradients that came
//
// Bound by the logits' bytes: one pass forward, one more (and the gradient written) backward.  A thread keeps its own
// running m, s and w over vectors of 16 bytes, four in flight, so that nothing passes between threads before a block's end.
// Rows that are fewer than the device has room for are split over blocks, whose sums the last one to arrive joins in block
// order (results repeat bit for bit).
//
// The best k of a row come from the same pass.  A block goes through its part in chunks of what its threads hold in
// registers.  The k-th largest of the threads' best values bounds the chunk's k-th largest from below, and at most
// k threads hold anything above it, so few values are candidates: they go to shared memory beside the best so far and are
// ranked by counting.  A logit and its index make one 64-bit key, larger for the larger logit and then for the lower
// index, so no two are equal and no order of arrival matters.

#include <algorithm>

#include "lq_internal.h"
#include "lq_tma.cuh"
#include "lq_common.cuh"

namespace lq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;                     // 16-byte loads of a thread in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -150.f;               // e^kFar is 0: what infinitely improbable logits are held at

struct LogprobParams {
    const void* x;
    int64_t stride;
    const int64_t* tokens;
    float *logprob, *entropy, *lse;
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

// Value `i` of a 16-byte vector.
template <class T>
__device__ __forceinline__ float value_of(const uint4& v, int i);
template <>
__device__ __forceinline__ float value_of<float>(const uint4& v, int i) { return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w); }
template <>
__device__ __forceinline__ float value_of<__half>(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return half_bits_to_float((uint16_t)(i & 1 ? w >> 16 : w));
}
template <>
__device__ __forceinline__ float value_of<__nv_bfloat16>(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}

// The aligned vector of values a .. a + VEC - 1 of a row of V values (a may be negative); -inf outside the row.  Only the
// vectors at a row's ends are read value by value, so nothing outside the row is touched.
template <class T, int VEC>
__device__ __forceinline__ void load_values(const T* row, int64_t a, int V, float (&x)[VEC]) {
    if (a >= 0 && a + VEC <= V) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + a);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = value_of<T>(v, i);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = a + i >= 0 && a + i < V ? to_float(row[a + i]) : -INFINITY;
    }
}

// Orders like the values (NaN above all, -0 as 0); never 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = x != x ? 0x7fc00000u : __float_as_uint(x + 0.f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o); }

// Low bits of an ordered value that say nothing: all 0, or all 1 below the order of 0.
template <class T>
struct LowBits {
    static constexpr int value = 0;
};
template <>
struct LowBits<__half> {
    static constexpr int value = 13;
};
template <>
struct LowBits<__nv_bfloat16> {
    static constexpr int value = 16;
};

struct Sums {
    float m, s, w;
};
// Both about one maximum.
__device__ __forceinline__ Sums joined(Sums a, Sums b) {
    const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.f : m;
    const float da = max_nan(a.m - ref, kFar), db = max_nan(b.m - ref, kFar);
    const float ea = ex2f(da * kLog2e), eb = ex2f(db * kLog2e);
    return Sums{m, a.s * ea + b.s * eb, (a.w + a.s * da) * ea + (b.w + b.s * db) * eb};
}

template <int VEC, int TOP>
struct Shared {
    static constexpr int kHeld = kVecs * VEC;                   // values of a thread
    static constexpr int kRoom = TOP ? TOP * kHeld + TOP : 1;   // candidates of a chunk, and the best so far
    unsigned long long found[kRoom], best[TOP ? TOP : 1];
    Sums sums[kWarps];
    int count, last;
};

// The `top` largest of `n` keys in found[] to best[], largest first (0 where there are fewer).  All threads call it.
template <int VEC, int TOP>
__device__ __forceinline__ void rank_keys(Shared<VEC, TOP>& S, int n, int top) {
    __syncthreads();
    for (int i = threadIdx.x; i < top; i += kThreads) S.best[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long mine = S.found[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += S.found[j] > mine;
        if (mine && above < top) S.best[above] = mine;
    }
    __syncthreads();
}

// TOP: the largest k this variant has room for, 0: no alternatives.
template <class T, int TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobParams P) {
    constexpr int VEC = 16 / sizeof(T), kChunk = kThreads * kVecs * VEC;
    constexpr int kLow = LowBits<T>::value;
    __shared__ Shared<VEC, TOP> S;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / P.splits, split = blockIdx.x - row * P.splits, V = P.V, top = P.top;
    const T* x = static_cast<const T*>(P.x) + row * P.stride;
    // chunks count from the 16-byte boundary at or before the row's first value
    const int before = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int chunks = (int)(((int64_t)V + before + kChunk - 1) / kChunk);
    const int c0 = (int)((int64_t)chunks * split / P.splits), c1 = (int)((int64_t)chunks * (split + 1) / P.splits);

    Sums mine{-INFINITY, 0.f, 0.f};
    if (TOP) {
        for (int i = tid; i < top; i += kThreads) S.best[i] = 0;
        if (tid == 0) S.count = 0;
        __syncthreads();
    }
    for (int c = c0; c < c1; ++c) {
        float v[kVecs][VEC];
        const int64_t at = (int64_t)c * kChunk - before + tid * VEC;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) load_values<T, VEC>(x, at + (int64_t)u * kThreads * VEC, V, v[u]);
        float m = mine.m;
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = fmaxf(m, v[u][i]);
        const float ref = m == -INFINITY ? 0.f : m;
        if (m != mine.m) {   // the sums so far about the new maximum
            const float d = max_nan(mine.m - ref, kFar), e = ex2f(d * kLog2e);
            mine.w = (mine.w + mine.s * d) * e;
            mine.s *= e;
            mine.m = m;
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = max_nan(v[u][i] - ref, kFar), e = ex2f(d * kLog2e);
                mine.s += e;
                mine.w = fmaf(e, d, mine.w);
            }
        if (TOP) {
            // this thread's best value, and what a value has to pass to matter
            uint32_t o = 0;
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int64_t j = at + (int64_t)u * kThreads * VEC + i;
                    if (j >= 0 && j < V) o = max(o, ordered(v[u][i]));
                }
            const uint32_t bar = (uint32_t)(S.best[top - 1] >> 32);   // (later values have higher indices: equal ones lose)
            int left = __syncthreads_count(o > bar);
            if (left == 0) continue;
            // t: the k-th largest of the threads' best, found bit by bit
            uint32_t least = bar + 1;
            bool mine_in = o > bar;
            if (left > top) {
                uint32_t t = 0;
                for (int b = 31; b >= kLow; --b) {
                    const uint32_t up = t | 1u << b;
                    if (__syncthreads_count(o >= up) >= top) t = up;
                }
                if (!(t >> 31)) t |= (1u << kLow) - 1u;
                least = max(least, t);
                const int above = __syncthreads_count(o > t);
                mine_in = o > t;
                // of the threads whose best is t those with the lowest index of one
                int first = kChunk;
                if (o == t) {
#pragma unroll
                    for (int u = kVecs - 1; u >= 0; --u)
#pragma unroll
                        for (int i = VEC - 1; i >= 0; --i) {
                            const int64_t j = at + (int64_t)u * kThreads * VEC + i;
                            if (j >= 0 && j < V && ordered(v[u][i]) == t) first = (u * kThreads + tid) * VEC + i;
                        }
                }
                int cut = kChunk - 1;   // the (top - above)-th smallest `first`
                if (__syncthreads_count(o == t) > top - above) {
                    int f = 0;
                    for (int b = 30 - __clz(kChunk); b >= 0; --b) {   // largest f with fewer than top - above below it
                        const int up = f | 1 << b;
                        if (__syncthreads_count(first < up) < top - above) f = up;
                    }
                    cut = f;
                }
                mine_in |= o == t && first <= cut;
            }
            if (mine_in) {
#pragma unroll
                for (int u = 0; u < kVecs; ++u)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int64_t j = at + (int64_t)u * kThreads * VEC + i;
                        const uint32_t k = ordered(v[u][i]);
                        if (j >= 0 && j < V && k >= least) S.found[atomicAdd(&S.count, 1)] = (unsigned long long)k << 32 | (0xffffffffu - (uint32_t)j);
                    }
            }
            __syncthreads();
            const int n = S.count;
            for (int i = tid; i < top; i += kThreads) S.found[n + i] = S.best[i];
            rank_keys(S, n + top, top);
            if (tid == 0) S.count = 0;   // (the next chunk's pushes come after its counting barrier)
        }
    }

    // ---- the block's sums ----
#pragma unroll
    for (int k = 16; k; k >>= 1) mine = joined(mine, Sums{__shfl_xor_sync(0xffffffffu, mine.m, k), __shfl_xor_sync(0xffffffffu, mine.s, k), __shfl_xor_sync(0xffffffffu, mine.w, k)});
    if (lane == 0) S.sums[warp] = mine;
    __syncthreads();
    Sums all = S.sums[0];
    for (int k = 1; k < kWarps; ++k) all = joined(all, S.sums[k]);
    if (P.splits > 1) {
        const int64_t slot = (int64_t)row * P.splits + split;
        if (tid < 3) P.part[3 * slot + tid] = tid == 0 ? all.m : tid == 1 ? all.s : all.w;
        if (TOP)
            for (int i = tid; i < top; i += kThreads) P.keys[slot * top + i] = S.best[i];
        __syncthreads();
        if (tid == 0) S.last = arrive(P.counters + row) == (unsigned)(P.splits - 1);
        __syncthreads();
        if (!S.last) return;
        if (tid == 0) P.counters[row] = 0;
        const float* p = P.part + 3 * (int64_t)row * P.splits;
        all = Sums{__ldcg(p), __ldcg(p + 1), __ldcg(p + 2)};
        for (int k = 1; k < P.splits; ++k) all = joined(all, Sums{__ldcg(p + 3 * k), __ldcg(p + 3 * k + 1), __ldcg(p + 3 * k + 2)});
        if (TOP) {
            const int n = P.splits * top;
            for (int i = tid; i < n; i += kThreads) S.found[i] = __ldcg(P.keys + (int64_t)row * P.splits * top + i);
            rank_keys(S, n, top);
        }
    }
    // ---- the row's results ----
    const float ref = all.m == -INFINITY ? 0.f : all.m, ln = logf(all.s);
    const bool none = all.s == 0.f;          // no token is possible
    if (TOP)
        for (int i = tid; i < top; i += kThreads) {
            const unsigned long long k = S.best[i];
            P.top_ids[(int64_t)row * top + i] = (int64_t)(0xffffffffu - (uint32_t)k);
            P.top_logprobs[(int64_t)row * top + i] = none ? -INFINITY : unordered((uint32_t)(k >> 32)) - ref - ln;
        }
    if (tid == 0) {
        if (P.entropy) P.entropy[row] = none ? 0.f : ln - all.w / all.s;
        if (P.lse) P.lse[row] = none ? -INFINITY : ref + ln;
        const int64_t t = P.tokens[row];
        if (t >= V) atomicOr(P.status, kStatusIndex);
        P.logprob[row] = t < 0 || t >= V ? 0.f : none ? -INFINITY : to_float(x[t]) - ref - ln;
    }
}

struct GradParams {
    const void* x;
    int64_t stride;
    void* dx;
    int64_t dx_stride;
    const int64_t* tokens;
    const float *lse, *entropy, *d_logprob, *d_entropy;
    int n, V, splits;
};

// Blocks of a row take its vectors in turn.
template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(const __grid_constant__ GradParams P) {
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
    const float lse = P.lse[row], ref = lse == -INFINITY ? 0.f : lse;
    const float g = given && P.d_logprob ? P.d_logprob[row] : 0.f;
    const float h = P.d_entropy ? P.d_entropy[row] : 0.f, H = h != 0.f ? P.entropy[row] : 0.f;
    const float c = -g - h * H;
    const int64_t step = (int64_t)P.splits * kThreads * VEC;
    for (int64_t a0 = ((int64_t)split * kThreads + threadIdx.x) * VEC - before; a0 < V; a0 += kVecs * step) {
        float v[kVecs][VEC];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) load_values<T, VEC>(x, a0 + u * step, V, v[u]);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int64_t a = a0 + u * step;
            alignas(16) T y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = max_nan(v[u][i] - ref, kFar), p = ex2f(d * kLog2e);
                const float r = p * fmaf(-h, d, c);
                y[i] = (T)(a + i == t ? r + g : r);
            }
            if (alike && a >= 0 && a + VEC <= V) *reinterpret_cast<uint4*>(dx + a) = *reinterpret_cast<const uint4*>(y);
            else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (a + i >= 0 && a + i < V) dx[a + i] = y[i];
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
    return P.top <= 8 ? run<T, 8>(P, stream) : P.top <= 32 ? run<T, 32>(P, stream) : run<T, kMaxLogprobTop>(P, stream);
}

}  // namespace

lq_status launch_logprobs(lq_handle h, const lq_logprobs_args& a, cudaStream_t stream) {
    LogprobParams P = {};
    P.x = a.logits, P.stride = a.row_stride, P.tokens = a.tokens;
    P.logprob = a.logprob, P.entropy = a.entropy, P.lse = a.lse, P.top_ids = a.top_ids, P.top_logprobs = a.top_logprobs;
    P.n = a.n, P.V = a.vocab, P.top = a.top;
    P.status = h->status_flag;
    // as many blocks of a row as let the device hold eight of all rows on each SM, a chunk or more each
    const int e = a.dtype == LQ_F32 ? 4 : 2, chunk = kThreads * kVecs * 16 / e;
    const int64_t want = std::max<int64_t>(1, (int64_t)h->num_sms * 8 / a.n);
    int64_t splits = std::min<int64_t>(want, ((int64_t)a.vocab + chunk - 1) / chunk);
    // (what the last block of a row joins fits its shared memory)
    if (a.top) splits = std::min<int64_t>(splits, 16 / e * kVecs);
    const size_t key_bytes = (size_t)a.n * splits * a.top * 8, bytes = key_bytes + (size_t)a.n * splits * 12;
    if (splits > 1 && ((size_t)a.n > h->num_counters || bytes > h->partial_floats * sizeof(float))) splits = 1;
    P.splits = (int)splits;
    P.keys = reinterpret_cast<unsigned long long*>(h->partials);
    P.part = h->partials + key_bytes / sizeof(float);
    P.counters = h->counters;
    if (a.dtype == LQ_F32) return run_top<float>(P, stream);
    return a.dtype == LQ_F16 ? run_top<__half>(P, stream) : run_top<__nv_bfloat16>(P, stream);
}

lq_status launch_logprobs_grad(lq_handle h, const lq_logprobs_grad_args& a, cudaStream_t stream) {
    GradParams P = {};
    P.x = a.logits, P.stride = a.row_stride, P.dx = a.d_logits, P.dx_stride = a.d_row_stride, P.tokens = a.tokens;
    P.lse = a.lse, P.entropy = a.entropy, P.d_logprob = a.d_logprob, P.d_entropy = a.d_entropy;
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
