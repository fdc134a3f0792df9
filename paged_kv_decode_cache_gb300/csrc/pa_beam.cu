// Beam search's selection: the K best continuations of every request over its
// beams and the vocabulary, in one launch that reads the logits once.
//
//   score(w, v) = cum_w + (x_wv - lse_w),  lse_w = max + ln sum_v exp(x_wv - max)
//
// Within a row the scores are ordered as the logits, so one pass over a
// row's logits gives both its (max, sum) and its K largest logits; lse enters
// only when the rows of a request are joined.  A CTA takes a slice of a row, in chunks
// of 4 16-byte vectors per thread; a thread's part of a chunk is a group.  The
// stream itself only sums and notes each group's maximum: it has no branch and
// no barrier.  After up to 16 chunks, what K of the threads' maxima reach bounds
// the K-th largest value from below, and only the groups that reach it (about twice K) are
// read again, from L2, for the values themselves.  (Taking candidates out
// while streaming cost as much again: 62 us against 32 for 256 rows of 151937 in
// bf16.)  The last CTA of a request to finish joins its lists.  Those rows now take
// 29 us: the stream 17 (4.5 TB/s: one wave of CTAs, which all start and end at once;
// L2 prefetches and deeper rings made it slower), 6 for the candidates, 4 for
// the join and 2 for the launch; 4 rows of 32000 take 8.4, a chain of latencies.
//
// Sums: 2^(k x - k max) in fp32 with one rounding of the exponent, k = log2 e in
// fp32, by which lse is divided in the end (exponent_unit); fp32 sums of 8 per vector and of a
// thread's vectors, 64 bits across threads and slices, the logarithm in fp32: an lse is
// good to 2^-19.  Scores are formed and compared in 64 bits, so that candidates of one beam
// keep their logits' order however large its score is (rounded to fp32 they could trade
// places); those of different beams can, within their lses' error.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                      // 16-byte vectors per thread and chunk
constexpr int kChunkVecs = kThreads * kVecs;
constexpr int kWarpVecs = 32 * kVecs;
constexpr int kStages = 2;                    // chunks of a warp's ring
constexpr int kGroupBytes = 8192;             // the groups' maxima between two looks for candidates
constexpr int kGroups = 256;                  // groups that a look can take
constexpr int kRingBytes = kThreads / 32 * kStages * (kWarpVecs + 1) * 16;
constexpr int kMaxK = 64;
constexpr int kMaxBeams = 64;
constexpr int kMaxJoin = 4096;                // candidates a request's join holds
constexpr int kJoinBytes = 20;                // of shared memory per candidate of a join
constexpr int kDirect = 128;                  // entries that a join ranks without a bound first
constexpr int kHeads = 1024;                  // lists' first entries that make the bound
// a score's two roundings in fp32, and its lse's: within 2^-24 of |cum| + |x| + |lse| each
constexpr float kSlack = 4.76837158e-7f;      // 2^-21
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPool = 2 * kThreads;            // candidates of a slice at a time
constexpr int kWaveCtas = 4 * 152;            // slices: one wave of 4 CTAs per SM
// Requests of one launch, and tickets at the workspace's start: their place is the same
// for every shape, so no call's lists ever lie where another's tickets are.
constexpr int kMaxTickets = 4096;

template <int N>
struct Int {
    static constexpr int value = N;
};

template <typename T>
struct Vec {  // a 16-byte vector of logits
    static constexpr int kElems = 16 / sizeof(T);
    static constexpr bool k16 = sizeof(T) == 2;
    // bits of the order-preserving key that a value can differ in: the top ones
    static constexpr int kKeyLow = k16 ? 16 : 0;
    static constexpr uint32_t kFill = k16 ? 0xff80ff80u : 0xff800000u;  // -inf
    __device__ static float get(const uint4 &v, int e) {
        const uint32_t w = (&v.x)[k16 ? e >> 1 : e];
        if constexpr (k16) return e & 1 ? bf16hi(w) : bf16lo(w);
        else return __uint_as_float(w);
    }
    __device__ static void put(uint32_t (&w)[4], int e, T x) {
        if constexpr (k16) {
            const uint32_t u = __bfloat16_as_ushort(x);
            w[e >> 1] = e & 1 ? (w[e >> 1] & 0x0000ffffu) | u << 16 : (w[e >> 1] & 0xffff0000u) | u;
        } else {
            w[e] = __float_as_uint(x);
        }
    }
    __device__ static float max(const uint4 (&v)[kVecs]) {
        if constexpr (k16) {
            auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
            __nv_bfloat162 m = h(v[0].x);
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                m = __hmax2(__hmax2(m, __hmax2(h(v[j].x), h(v[j].y))), __hmax2(h(v[j].z), h(v[j].w)));
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            float m = get(v[0], 0);
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                m = fmaxf(fmaxf(m, fmaxf(get(v[j], 0), get(v[j], 1))), fmaxf(get(v[j], 2), get(v[j], 3)));
            return m;
        }
    }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float &d, float x) { d = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }

// Order-preserving map of a float (no NaN; -0 as +0) to an unsigned integer, and back.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// (16-bit values: the key's low half, left 0 by the search, is all ones in a negative value's key)
template <int kKeyLow>
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~(k | ((1u << kKeyLow) - 1u)));
}
__device__ __forceinline__ uint64_t order_key(double x) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k & ~(1ull << 63) : ~k));
}

// A candidate of a slice as one number: its logit's order, then the lower
// vocabulary entry first.  0: none.
__device__ __forceinline__ uint64_t candidate(float x, int v) {
    return static_cast<uint64_t>(order_key(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(v));
}
__device__ __forceinline__ float candidate_value(uint64_t c) {
    const uint32_t k = static_cast<uint32_t>(c >> 32);
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ int candidate_entry(uint64_t c) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(c)); }

struct BeamArgs {
    float *scores;
    int32_t *tokens, *parents;
    const void *logits;
    int64_t row_stride;
    const float *cum;
    const uint8_t *finished;
    int32_t eos;
    int beams, vocab, K, slices;
    int32_t row0;          // this launch's first row of the call
    int32_t *tickets;      // [kMaxTickets], zero between calls
    float *part_max;       // [rows, slices]
    double *part_sum;      // [rows, slices]
    uint64_t *part_list;   // [rows, slices, K] candidates
};

// A row's vectors: vector i holds entries i E .. i E + E - 1, whatever the row's
// alignment, so that equal rows give equal sums to the last bit.  A row that starts
// `skew` bytes past a 16-byte boundary takes each vector from two aligned ones.
//
// Warp w's share of a chunk is vectors c0 + w kWarpVecs + j 32 + lane (j < kVecs),
// which it streams through its own ring in shared memory, a chunk ahead (cp.async;
// only the warp waits for it): 64 KB in flight per SM throughout.
template <typename T>
struct Row {
    static constexpr int E = Vec<T>::kElems;
    const T *x;
    const uint4 *grid;
    int skew, vocab;
    int whole;   // vectors below it lie (both aligned halves) inside the row

    __device__ Row(const T *row, int n) : x(row), vocab(n) {
        skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
        grid = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(x) - skew);
        whole = skew ? (vocab + skew / static_cast<int>(sizeof(T))) / E - 1 : vocab / E;
    }
    // This warp's share of the chunk at c0 (vectors below `end`) on its way to `slot`.
    __device__ __forceinline__ void fetch(uint4 *slot, int c0, int end) const {
        const int lane = threadIdx.x & 31, first = c0 + static_cast<int>(threadIdx.x >> 5) * kWarpVecs;
        int stop = min(end, whole);        // aligned vectors needed
        stop += skew && stop > 0 ? 1 : 0;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = j * 32 + lane;
            if (first + i < stop) cp_async_16(slot + i, grid + first + i);
        }
        if (lane == 0 && skew && first + kWarpVecs < stop) cp_async_16(slot + kWarpVecs, grid + first + kWarpVecs);
    }
    template <int W>
    __device__ __forceinline__ void take_skewed(uint4 (&raw)[kVecs], const uint4 *slot) const {  // skew = 4 W + (0 or 2)
        const int lane = threadIdx.x & 31, bits = (skew & 3) * 8;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const uint4 lo = slot[j * 32 + lane], hi = slot[j * 32 + lane + 1];
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            raw[j] = make_uint4(__funnelshift_r(w[W], w[W + 1], bits), __funnelshift_r(w[W + 1], w[W + 2], bits),
                                __funnelshift_r(w[W + 2], w[W + 3], bits), __funnelshift_r(w[W + 3], w[W + 4], bits));
        }
    }
    // The chunk's vectors of this thread, fetched before: -inf past the end, and
    // the row's end entry by entry.
    __device__ __forceinline__ void take(uint4 (&raw)[kVecs], const uint4 *slot, int c0, int end) const {
        using V = Vec<T>;
        if (skew == 0) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) raw[j] = slot[j * 32 + (threadIdx.x & 31)];
        } else if (skew < 4) {
            take_skewed<0>(raw, slot);
        } else if (skew < 8) {
            take_skewed<1>(raw, slot);
        } else if (skew < 12) {
            take_skewed<2>(raw, slot);
        } else {
            take_skewed<3>(raw, slot);
        }
        if (c0 + kChunkVecs <= min(end, whole)) return;   // (the same for the CTA)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = vector_of(c0, j);
            if (i < end && i < whole) continue;
            raw[j] = make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
            if (i >= end) continue;
            uint32_t w[4] = {V::kFill, V::kFill, V::kFill, V::kFill};
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (i * E + e < vocab) V::put(w, e, x[i * E + e]);
            raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ static int vector_of(int c0, int j) {
        return c0 + static_cast<int>(threadIdx.x >> 5) * kWarpVecs + j * 32 + static_cast<int>(threadIdx.x & 31);
    }
};

// A key that at least K of the threads' keys reach (0: fewer than K are not 0).
// The ceil(K / warps)-th largest of each of the first `warps` warps, and the lowest of
// those: two barriers, and for values in no order about twice as many keys reach it as
// the K-th largest.  Where a warp has too few keys, or values that rise along the row let far more
// reach it, the K-th largest, bit by bit from the top with a CTA-wide count per bit.
template <int kKeyLow>
__device__ __forceinline__ uint32_t reached_by(uint32_t mine, int K, uint32_t *warp_keys, int warps = kThreads / 32) {
    const int lane = threadIdx.x & 31;
    uint32_t left = mine, best = 0;
    for (int r = (K + warps - 1) / warps; r > 0; --r) {
        best = __reduce_max_sync(0xffffffffu, left);
        const uint32_t who = __ballot_sync(0xffffffffu, left == best);
        if (lane == __ffs(who) - 1) left = 0;
    }
    if (lane == 0) warp_keys[threadIdx.x >> 5] = best;
    __syncthreads();
    uint32_t key = warp_keys[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) key = min(key, i < warps ? warp_keys[i] : key);
    if (__syncthreads_count(key && mine >= key) <= 3 * K + 16 && key) return key;
    key = 0;
    for (int bit = 31; bit >= kKeyLow; --bit)
        if (__syncthreads_count(mine >= (key | 1u << bit)) >= K) key |= 1u << bit;
    return key;
}

// A sum with maximum m holds 2^(u x - u m), with u = k, and u m the product ROUNDED, at
// every place the same number.  (Contracted into an fma it would be another one, off by
// up to 2^-24 of itself: 0.003 in a score at logits of 60000.)  The terms carry the
// product's rounding as a factor, which from 2^31 on could leave fp32's range (rows
// masked with -1e30 or with the type's lowest value).  Beyond 2^30 therefore u = 1/2,
// whose products are exact: values there are 128 apart or more, so that in either
// unit only those equal to m count.
constexpr float kFar = 0x1p30f;
__device__ __forceinline__ float exponent_unit(float m) { return fabsf(m) <= kFar ? kLog2e : 0.5f; }

// By what a sum with maximum a is multiplied to count from b >= a.
__device__ __forceinline__ float ratio(float a, float b) {
    if (fmaxf(fabsf(a), fabsf(b)) > kFar) return a == b ? 1.f : 0.f;   // (-inf: its sum is 0 or NaN)
    return fast_exp2(__fsub_rn(__fmul_rn(a, kLog2e), __fmul_rn(b, kLog2e)));
}

// log2 z for a normal z as whole + the result, to 2^-23 or so, in integers and fp32: CUDA's
// log2(double) is a chain of some 60 FP64 instructions, 1 us here, which a GB300 SM
// issues at 1/64 of its FP32 rate.  z = 2^whole (m + r) with m, the first 24 bits, in
// [0.6875, 1.375).  NaN for a NaN.
__device__ __forceinline__ float log2_of_sum(double z, int *whole) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(z));
    const int up = (u >> 49 & 7) >= 3;   // 1.375 and above is halved
    *whole = static_cast<int>(u >> 52) - 1023 + up;
    const float m = __uint_as_float(static_cast<uint32_t>(127 - up) << 23 | (static_cast<uint32_t>(u >> 29) & 0x7fffffu));
    const float r = static_cast<float>(static_cast<uint32_t>(u) & 0x1fffffffu) * (up ? 0x1p-53f : 0x1p-52f);
    return u >> 52 < 0x7ff ? kLog2e * (logf(m) + r / m) : NAN;
}

// Sum of f(j) over j in [0, n) by a team of 2^t threads; every thread of the CTA calls.
template <typename F>
__device__ __forceinline__ int team_sum(int n, int t, F &&f) {
    int sum = 0;
#pragma unroll 8
    for (int j = threadIdx.x & ((1 << t) - 1); j < n; j += 1 << t) sum += f(j);
    for (int o = 1 << t >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
// log2 of the CTA's threads for each of n entries: a power of two, at most a warp.
__device__ __forceinline__ int team_of(int n) {
    static_assert(kThreads == 256, "8 - t: entries of teams of 2^t");
    return n <= 8 ? 5 : max(0, 8 - (32 - __clz(n - 1)));
}

// How many of pool[0 .. n) come before c; four at a time, so the pool has room for 3
// more entries, which the caller has set to 0.
__device__ __forceinline__ int place_of(uint64_t c, const uint64_t *pool, int n) {
    int place = 0;
#pragma unroll 2
    for (int j = 0; j < n; j += 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(pool + j);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(pool + j + 2);
        place += (a.x > c) + (a.y > c) + (b.x > c) + (b.y > c);
    }
    return place;
}

// pool[0 .. n) reduced to its min(n, K) first candidates, in order: an entry's
// place is the number of entries before it.  n <= kPool = 2 kThreads.
__device__ __noinline__ int keep_first(uint64_t *pool, int n, int K) {
    if (threadIdx.x < 3) pool[n + threadIdx.x] = 0;
    __syncthreads();
    uint64_t c[2];
    int place[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = u * kThreads + threadIdx.x;
        place[u] = K;
        if (i < n) {
            c[u] = pool[i];
            place[u] = place_of(c[u], pool, n);
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (place[u] < K) pool[place[u]] = c[u];
    __syncthreads();
    return min(n, K);
}

// The K first candidates of vectors [v0, v1) whatever their order: for rows
// that overfill the pool (long runs of equal values, or values that rise along the
// row).  Each chunk's exact K-th largest value by bisection over its key, then, among
// the values equal to it, the lowest entries by bisection over the entry.
// pool: the list so far in [0, kept), the chunk's share after it.
template <typename T>
__device__ __noinline__ int exact_slice(const Row<T> &row, int v0, int v1, int K, uint64_t *pool, int *count,
                                        uint4 *slot) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    const int tid = threadIdx.x;
    int kept = 0;
    float floor = -INFINITY;   // values at or below it are not among the K largest
    for (int c0 = v0; c0 < v1; c0 += kChunkVecs) {
        uint4 raw[kVecs];
        __syncwarp();
        row.fetch(slot, c0, v1);
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        row.take(raw, slot, c0, v1);
        auto each = [&](auto &&f) {  // f(value, vocabulary entry) of this thread's values above the floor
            for (int j = 0; j < kVecs; ++j)
                for (int e = 0; e < E; ++e) {
                    const float v = V::get(raw[j], e);
                    if (v > floor) f(v, Row<T>::vector_of(c0, j) * E + e);
                }
        };
        auto total = [&](auto &&pred) {
            __syncthreads();
            if (tid == 0) *count = 0;
            __syncthreads();
            int c = 0;
            each([&](float v, int i) { c += pred(v, i); });
            c = __reduce_add_sync(0xffffffffu, c);
            if ((tid & 31) == 0 && c) atomicAdd(count, c);
            __syncthreads();
            return *count;
        };
        const int above = total([](float, int) { return 1; });
        if (above == 0) continue;
        float kth = floor;   // with fewer than K above the floor, all of them
        int last = -1;       // the highest entry of a value equal to it that is taken
        if (above > K) {
            uint32_t key = 0u;
            for (int bit = 31; bit >= V::kKeyLow; --bit) {
                const uint32_t t = key | 1u << bit;
                if (total([&](float v, int) { return order_key(v) >= t; }) >= K) key = t;
            }
            kth = key_value<V::kKeyLow>(key);
            const int need = K - total([&](float v, int) { return v > kth; });
            last = 0;
            for (int bit = 30; bit >= 0; --bit) {
                const int t = last | 1 << bit;
                if (total([&](float v, int i) { return v == kth && i < t; }) < need) last = t;
            }
        }
        __syncthreads();
        if (tid == 0) *count = kept;
        __syncthreads();
        each([&](float v, int i) {
            if (!(v > kth || (v == kth && i <= last))) return;
            const int at = atomicAdd(count, 1);
            if (at < kPool) pool[at] = candidate(v, i);
        });
        __syncthreads();
        kept = keep_first(pool, min(*count, kPool), K);
        if (kept == K) floor = candidate_value(pool[K - 1]);
    }
    return kept;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamArgs a) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    extern __shared__ __align__(16) uint64_t dyn_smem[];  // the warps' rings; then kJoinBytes per entry of the join
    __shared__ uint32_t warp_keys[kThreads / 32];
    __shared__ __align__(16) uint64_t pool[kPool + 4];  // candidates for the slice's K largest
    __shared__ int count, groups, ticket;
    constexpr int kBatch = kGroupBytes / (kThreads * static_cast<int>(sizeof(T)));   // chunks: 16 (fp32: 8)
    __shared__ T group_max[kBatch * kThreads];               // [kBatch][kThreads], exact in T
    __shared__ int group_at[kGroups];
    __shared__ float red_max[kThreads / 32];
    __shared__ double red_sum[kThreads / 32];
    __shared__ double lse[kMaxBeams];
    __shared__ float beam_cum[kMaxBeams], base[kMaxBeams], slack[kMaxBeams], head[kMaxBeams];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_id = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
    const int group = row_id / a.beams, K = a.K;
    const int first_row = group * a.beams;
    const Row<T> row(static_cast<const T *>(a.logits) + row_id * a.row_stride, a.vocab);
    const int vecs = (a.vocab + E - 1) / E;
    const int per = (vecs + a.slices - 1) / a.slices;
    const int v0 = min(slice * per, vecs), v1 = min(v0 + per, vecs);
    uint4(*ring)[kWarpVecs + 1] = reinterpret_cast<uint4(*)[kWarpVecs + 1]>(
        reinterpret_cast<uint4 *>(dyn_smem) + warp * kStages * (kWarpVecs + 1));   // [kStages], this warp's
#pragma unroll
    for (int u = 0; u < kStages - 1; ++u) {   // (on its way before `finished` is looked at)
        if (v0 + u * kChunkVecs < v1) row.fetch(ring[u], v0 + u * kChunkVecs, v1);
        cp_async_commit();
    }
    const bool done = a.finished && a.finished[row_id];
    if (tid < a.beams) beam_cum[tid] = a.cum[first_row + tid];   // (for the join, which would wait for them)

    const int64_t part = static_cast<int64_t>(row_id) * a.slices + slice;
    if (done) {   // its one continuation, as the only entry of a row with lse = 0
        cp_async_wait<0>();
        if (tid == 0) {
            a.part_max[part] = slice == 0 ? 0.f : -INFINITY;
            a.part_sum[part] = slice == 0 ? 1.0 : 0.0;
        }
        if (tid < K) a.part_list[part * K + tid] = slice == 0 && tid == 0 ? candidate(0.f, a.eos) : 0;
    } else {
        float m = -INFINITY;              // this thread's maximum
        float unit = kLog2e, minus = 0.f; // (a NaN goes into the sum all the same)
        uint64_t sum2 = 0;                // and sum of 2^(x k - m k), in two halves
        float floor = -INFINITY;          // values at or below it are not among the slice's K largest
        bool overfull = false;
        int kept = 0;                     // the K largest so far, pool[0 .. kept)
        int stage = 0;
        for (int b0 = v0; b0 < v1; b0 += kBatch * kChunkVecs) {
            const int b1 = min(b0 + kBatch * kChunkVecs, v1);
            // ---- stream: sums, and each thread's maximum of each chunk
            float bmax = -INFINITY;
            T *gmax = group_max + tid;
            for (int c0 = b0; c0 < b1; c0 += kChunkVecs, gmax += kThreads) {
                const int next = c0 + (kStages - 1) * kChunkVecs;
                if (next < v1) row.fetch(ring[stage ? stage - 1 : kStages - 1], next, v1);
                cp_async_commit();
                cp_async_wait<kStages - 1>();
                __syncwarp();    // (every lane's copies of this chunk have landed)
                uint4 raw[kVecs];
                row.take(raw, ring[stage], c0, v1);
                __syncwarp();    // (and are read: the next fetch may go there)
                stage = stage == kStages - 1 ? 0 : stage + 1;
                const float cmax = V::max(raw);
                from_float(*gmax, cmax);
                bmax = fmaxf(bmax, cmax);
                if (cmax > m) {
                    const float f = ratio(m, cmax);   // (m = -inf: 0)
                    sum2 = mul2(sum2, pack2(f, f));
                    m = cmax;
                    unit = exponent_unit(m);
                    minus = -__fmul_rn(m, unit);
                }
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    uint64_t two[E / 2];
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        float a0, a1;
                        unpack2(fma2(pack2(V::get(raw[j], e), V::get(raw[j], e + 1)), pack2(unit, unit),
                                     pack2(minus, minus)), a0, a1);
                        two[e / 2] = pack2(fast_exp2(a0), fast_exp2(a1));
                    }
#pragma unroll
                    for (int o = E / 4; o > 0; o >>= 1)
#pragma unroll
                        for (int e = 0; e < o; ++e) two[e] = add2(two[e], two[e + o]);
                    sum2 = add2(sum2, two[0]);
                }
            }
            // ---- the groups (a thread's values of a chunk) that may hold one of the K largest
            // (a short slice fills the first warps only; the last of them counts if it can give its share)
            const int full = min((b1 - b0) / kWarpVecs, kThreads / 32), rest = b1 - b0 >= kChunkVecs ? 0 : (b1 - b0) % kWarpVecs;
            const int warps = max(1, full + (min(rest, 32) * (full + 1) >= K ? 1 : 0));
            const uint32_t key = reached_by<V::kKeyLow>(bmax > floor ? order_key(bmax) : 0u, K, warp_keys, warps);
            const float cut = key ? key_value<V::kKeyLow>(key) : floor;
            const bool strict = key == 0;   // (fewer than K threads have any value above the floor: all such values)
            if (tid == 0) groups = 0, count = kept;
            __syncthreads();
            if (bmax > floor && (strict ? bmax > cut : bmax >= cut)) {
                gmax = group_max + tid;
                for (int c0 = b0; c0 < b1; c0 += kChunkVecs, gmax += kThreads)
                    if (strict ? to_float(*gmax) > cut : to_float(*gmax) >= cut) {
                        const int at = atomicAdd(&groups, 1);
                        if (at < kGroups) group_at[at] = Row<T>::vector_of(c0, 0);   // its first vector
                    }
            }
            __syncthreads();
            const int n_groups = groups;
            if (n_groups > kGroups) overfull = true;
            // ---- a warp per group: its values again, now from L2 (four groups' on their way at once)
            static_assert(kVecs * E <= 32, "a group's values, one per lane");
            constexpr int kAtOnce = 4, kWarps = kThreads / 32;
            const int found = min(n_groups, kGroups);
            for (int g0 = warp; g0 < found; g0 += kAtOnce * kWarps) {
                float value[kAtOnce];
                int entry[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int g = g0 + u * kWarps, v = group_at[min(g, kGroups - 1)] + lane / E * 32;
                    entry[u] = v * E + lane % E;
                    value[u] = g < found && lane < kVecs * E && v < v1 && entry[u] < a.vocab ? to_float(row.x[entry[u]])
                                                                                             : -INFINITY;
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u)
                    if (strict ? value[u] > cut : value[u] >= cut) {
                        const int at = atomicAdd(&count, 1);
                        if (at < kPool) pool[at] = candidate(value[u], entry[u]);
                    }
            }
            __syncthreads();
            if (count > kPool) overfull = true;
            if (overfull) {
                kept = 0, floor = INFINITY;   // (the sums go on; the list is made again below)
                __syncthreads();
                continue;
            }
            kept = keep_first(pool, count, K);
            if (kept == K) floor = candidate_value(pool[K - 1]);   // (later entries of an equal value come after it)
        }
        __syncthreads();
        if (overfull) kept = exact_slice<T>(row, v0, v1, K, pool, &count, ring[0]);
        // ---- the slice's maximum, sum and list
        float sum, sum_odd, top = m;
        unpack2(sum2, sum, sum_odd);
        sum += sum_odd;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) red_max[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, red_max[i]);
        double z = sum * ratio(m, top);  // (m = -inf: 0 or NaN)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) red_sum[warp] = z;
        __syncthreads();
        if (tid == 0) {
            static_assert(kThreads == 256, "eight warps' sums");
            a.part_max[part] = top;
            a.part_sum[part] = ((red_sum[0] + red_sum[1]) + (red_sum[2] + red_sum[3])) +
                               ((red_sum[4] + red_sum[5]) + (red_sum[6] + red_sum[7]));
        }
        if (tid < K) a.part_list[part * K + tid] = tid < kept ? pool[tid] : 0;
    }

    // ---- the request's last CTA joins its rows' slices
    __syncthreads();
    if (tid == 0) {   // (the fences of one thread, behind and before the CTA's barriers, order all its threads' accesses)
        __threadfence();
        ticket = atomicAdd(a.tickets + group, 1);
        __threadfence();
    }
    __syncthreads();
    if (ticket != a.beams * a.slices - 1) return;
    if (tid == 0) a.tickets[group] = 0;
    // ---- everything the slices left, in one round trip
    const int lists = a.beams * a.slices, entries = lists * K;
    uint64_t *keys = dyn_smem;                                      // [entries] candidates
    uint64_t *top_keys = keys + entries;                            // [entries] scores' keys, of those that the bound leaves
    int *top_index = reinterpret_cast<int *>(top_keys + entries);   // [entries] place in beams x vocabulary
    double *slice_sum = reinterpret_cast<double *>(top_keys);       // [lists], then the maxima
    float *slice_max = reinterpret_cast<float *>(top_index);        // [lists]
    const int64_t part0 = static_cast<int64_t>(first_row) * a.slices;
    for (int i = tid; i < entries; i += kThreads)
        keys[i] = __ldcg(reinterpret_cast<const unsigned long long *>(a.part_list) + part0 * K + i);
    for (int l = tid; l < lists; l += kThreads) {
        slice_max[l] = __ldcg(a.part_max + part0 + l);
        slice_sum[l] = __ldcg(a.part_sum + part0 + l);
    }
    if (tid == 0) count = 0;
    __syncthreads();
    // ---- the rows' lse, a few threads per row
    const int t_lse = a.slices > 16 ? 5 : 32 - __clz(a.slices - 1), team = 1 << t_lse;
    for (int w0 = 0; w0 < a.beams; w0 += kThreads >> t_lse) {
        const int w = w0 + (tid >> t_lse), first = w < a.beams ? tid & (team - 1) : a.slices;
        const float *of_max = slice_max + w * a.slices;
        const double *of_sum = slice_sum + w * a.slices;
        float M = -INFINITY;
        double z = 0.0;
        for (int i = first; i < a.slices; i += team) M = fmaxf(M, of_max[i]);
        for (int o = team >> 1; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        for (int i = first; i < a.slices; i += team)
            z += of_sum[i] * ratio(of_max[i], M);
        for (int o = team >> 1; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (first == 0 && w < a.beams) {
            int whole;
            const float part = log2_of_sum(z, &whole);
            // the maximum's product + whole + part, exact but for part's last bits, as two
            // floats; next to the range's ends the maximum itself stands beside them
            const bool far = exponent_unit(M) != kLog2e;
            const float ref = far ? 0.f : __fmul_rn(M, kLog2e);
            const float add = static_cast<float>(whole), top = ref + add, back = top - ref;
            const float low = ((ref - (top - back)) + (add - back)) + part;
            const float cum = beam_cum[w];
            head[w] = far ? M : 0.f;
            const float l = M > -INFINITY ? (top + low) * (1.f / kLog2e) + head[w] : INFINITY;
            lse[w] = M > -INFINITY ? (static_cast<double>(top) + low) * (1.0 / kLog2e) : INFINITY;
            base[w] = cum > -INFINITY && l < INFINITY ? fmaxf(cum - l, -FLT_MAX) : -INFINITY;   // (-inf: no candidates)
            slack[w] = kSlack * (fabsf(cum) + fabsf(l));
        }
    }
    __syncthreads();
    // ---- the candidates that may be among the K best: a score's range in fp32, what K
    // of the lower ends of the lists' first few reach, and 64 bits only
    // for those whose upper end reaches it.  (An SM's few FP64 units take some 250
    // cycles for one operation of every thread.)  Few candidates are all taken.
    auto range_of = [&](int w, uint64_t c, float &lo, float &hi) {
        if (c == 0 || !(base[w] > -INFINITY)) return false;
        const float x = candidate_value(c), s = fmaxf(x + base[w], -FLT_MAX), d = slack[w] + kSlack * fabsf(x);
        lo = d < INFINITY ? s - d : -INFINITY;
        hi = s + d;
        return true;
    };
    const int spread = lane * (kThreads / 32) + warp;   // (consecutive entries: one to a warp)
    const float per_entry = 1.f / (a.slices * K);       // (below 2^-12: (i + 0.5) times it is never near a whole number)
    float lo, hi;
    uint32_t bound = 0;
    if (entries > kDirect) {
        const int each = min(K, (kHeads + lists - 1) / lists);
        uint32_t mine = 0;
        for (int i = spread; i < lists * each; i += kThreads) {
            const int l = i / each;
            if (range_of(l / a.slices, keys[l * K + i % each], lo, hi)) mine = max(mine, order_key(lo));
        }
        bound = reached_by<0>(mine, K, warp_keys);
    }
    const float cut = bound ? key_value<0>(bound) : -INFINITY;
    for (int i = tid; i < entries; i += kThreads) {
        const int w = static_cast<int>((i + 0.5f) * per_entry);
        const uint64_t c = keys[i];
        if (!range_of(w, c, lo, hi) || !(hi >= cut)) continue;
        const double score = beam_cum[w] + ((candidate_value(c) - head[w]) - lse[w]);   // (in 64 bits)
        if (!(score > -INFINITY)) continue;
        const int at = atomicAdd(&count, 1);
        top_keys[at] = order_key(score);
        top_index[at] = w * a.vocab + candidate_entry(c);
    }
    __syncthreads();
    const int n = count, t = team_of(n);
    const int64_t out = static_cast<int64_t>(group) * K;
    for (int i0 = 0; i0 < n; i0 += kThreads >> t) {
        const int i = i0 + (tid >> t);
        const uint64_t k = i < n ? top_keys[i] : 0;
        const int at = i < n ? top_index[i] : 0;
        const int place = team_sum(n, t, [&](int j) {   // (no branch: short-circuits cost 50 ns per entry)
            return static_cast<int>(top_keys[j] > k) | (static_cast<int>(top_keys[j] == k) & static_cast<int>(top_index[j] < at));
        });
        if (i < n && place < K && (tid & ((1 << t) - 1)) == 0) {
            a.scores[out + place] = static_cast<float>(key_value(k));
            a.tokens[out + place] = at % a.vocab;
            a.parents[out + place] = a.row0 + first_row + at / a.vocab;
        }
    }
    for (int i = n + tid; i < K; i += kThreads) {  // fewer candidates than K
        a.scores[out + i] = -INFINITY;
        a.tokens[out + i] = -1;
        a.parents[out + i] = -1;
    }
}

int elem_size(int32_t type) { return type == PA_LOGITS_BF16 ? 2 : type == PA_LOGITS_F32 ? 4 : 0; }

// Slices of a row: no more CTAs than the GPU holds at once (256 rows: 2 slices take
// less than 3 to 5), each with at least a chunk.  A chunk more per slice costs a
// CTA about 0.4 us and 100 candidates more in the join 0.15, so of C chunks and
// beams x K candidates per slice, s^2 is about 300 C / (beams K); half of that, since
// CTAs that share an SM slow one another (64 rows of 151937, 8 beams, K = 16: 4
// slices 18 us, 9 slices 21; one request of them: 4 15.5, 6 16, 19 14.8).  And no more
// than the join holds.
int slices_of(int64_t rows, int beams, int vocab, int K, int elem) {
    const int64_t vecs = (static_cast<int64_t>(vocab) * elem + 15) / 16, chunks = (vecs + kChunkVecs - 1) / kChunkVecs;
    int64_t s = std::min(chunks, std::max<int64_t>(1, kWaveCtas / rows));
    while (s > 1 && s * s * beams * K > 150 * chunks) --s;
    s = std::min<int64_t>(s, kMaxJoin / (beams * K));
    return static_cast<int>(std::max<int64_t>(1, s));
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

bool shape_ok(int32_t groups, int32_t beams, int32_t vocab, int32_t K) {
    return groups >= 0 && beams > 0 && vocab > 0 && K > 0;
}
bool shape_supported(int32_t groups, int32_t beams, int32_t vocab, int32_t K) {
    return beams <= kMaxBeams && K <= kMaxK && static_cast<int64_t>(beams) * vocab <= INT32_MAX / 2 &&
           static_cast<int64_t>(groups) * beams <= (1 << 20);
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t vocab, int32_t K, int32_t logits_type) {
    if (!pa::shape_ok(groups, beams, vocab, K) || !pa::shape_supported(groups, beams, vocab, K) ||
        !pa::elem_size(logits_type) || groups == 0)
        return 0;
    const int64_t rows = static_cast<int64_t>(std::min<int32_t>(groups, pa::kMaxTickets)) * beams;
    // (fewer rows are cut into more slices: enough for them too)
    const int64_t most = rows * pa::slices_of(beams, beams, vocab, K, pa::elem_size(logits_type));
    const size_t parts = std::max(rows, std::min<int64_t>(most, pa::kWaveCtas));
    return 4 * pa::kMaxTickets + pa::up(4 * parts) + pa::up(8 * parts) + pa::up(8 * parts * K);
}

int pa_beam_select(float *scores, int32_t *tokens, int32_t *parents, const void *logits, int32_t logits_type,
                   int64_t row_stride, const float *cum, const uint8_t *finished, int32_t eos, int32_t groups,
                   int32_t beams, int32_t vocab, int32_t K, void *workspace, size_t workspace_bytes,
                   pa_stream_t stream) {
    if (!pa::shape_ok(groups, beams, vocab, K) || !pa::elem_size(logits_type) || row_stride < vocab) return PA_EINVAL;
    if (finished && (eos < 0 || eos >= vocab)) return PA_EINVAL;
    if (!pa::shape_supported(groups, beams, vocab, K)) return PA_EUNSUPPORTED;
    if (groups == 0) return PA_OK;
    if (!scores || !tokens || !parents || !logits || !cum) return PA_EINVAL;
    if (!pa::is_aligned(logits, 16) || !pa::is_aligned(scores, 4) || !pa::is_aligned(tokens, 4) ||
        !pa::is_aligned(parents, 4) || !pa::is_aligned(cum, 4))
        return PA_EINVAL;
    if (!workspace || workspace_bytes < pa_beam_workspace_bytes(groups, beams, vocab, K, logits_type) ||
        !pa::is_aligned(workspace, 256))
        return PA_EWORKSPACE;
    const int64_t rows = static_cast<int64_t>(std::min<int32_t>(groups, pa::kMaxTickets)) * beams;  // of a launch
    pa::BeamArgs a{};
    a.row_stride = row_stride, a.eos = eos;
    a.beams = beams, a.vocab = vocab, a.K = K;
    a.slices = pa::slices_of(rows, beams, vocab, K, pa::elem_size(logits_type));
    const size_t parts = static_cast<size_t>(rows) * a.slices;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.tickets = reinterpret_cast<int32_t *>(ws);
    ws += 4 * pa::kMaxTickets;
    a.part_max = reinterpret_cast<float *>(ws);
    ws += pa::up(4 * parts);
    a.part_sum = reinterpret_cast<double *>(ws);
    ws += pa::up(8 * parts);
    a.part_list = reinterpret_cast<uint64_t *>(ws);
    const int smem = std::max(pa::kRingBytes, beams * a.slices * K * pa::kJoinBytes);
    auto kern = logits_type == PA_LOGITS_BF16 ? pa::beam_select_kernel<__nv_bfloat16> : pa::beam_select_kernel<float>;
    static std::atomic<uint64_t> smem_attr_done[2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(smem_attr_done[logits_type].load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, pa::kMaxJoin * pa::kJoinBytes) != cudaSuccess)
            return PA_ECUDA;
        smem_attr_done[logits_type].fetch_or(bit, std::memory_order_release);
    }
    for (int32_t g0 = 0; g0 < groups; g0 += pa::kMaxTickets) {
        const int64_t r0 = static_cast<int64_t>(g0) * beams, n = std::min(groups - g0, pa::kMaxTickets);
        a.row0 = static_cast<int32_t>(r0);
        a.scores = scores + static_cast<int64_t>(g0) * K;
        a.tokens = tokens + static_cast<int64_t>(g0) * K;
        a.parents = parents + static_cast<int64_t>(g0) * K;
        a.logits = static_cast<const uint8_t *>(logits) + r0 * row_stride * pa::elem_size(logits_type);
        a.cum = cum + r0;
        a.finished = finished ? finished + r0 : nullptr;
        if (pa::launch_maybe_cooperative(kern, dim3(static_cast<unsigned>(n * beams * a.slices)), pa::kThreads, smem, stream,
                                         false, pa::pdl_on(), a) != cudaSuccess)
            return PA_ECUDA;
    }
    return PA_OK;
}

}  // extern "C"
