// Selection of the m largest of many keys by the CTAs of a thread-block cluster, for
// pa_blocks_select and pa_cache_evict: a row's keys are spread over the cluster's
// shared memory, a contiguous range per CTA, and stay there (pa_blocks_select's are all in
// one CTA's, and C = 1).
//
// cluster_narrow finds the m-th largest key by narrowing a range of key values: each
// pass counts the keys of the range in 2048 equal bins (shared-memory atomics in every
// CTA, the counts added up through distributed shared memory) and keeps the bin that
// holds the border.  The range starts at the keys' own least and largest, so keys of
// one sign and a few exponents are split finely by the first pass; 32-bit keys take at
// most 3.  A round trip through distributed shared memory costs most of a pass: every
// thread has all its loads of one in flight at once (one after the other, 7 CTAs'
// counts took 4 us a pass).
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kTopkBits = 11;
constexpr int kTopkBins = 1 << kTopkBits;
constexpr int kTopkFew = 64;   // keys that cluster_finish ranks, at most

// Larger floats have larger keys; -0 and 0 have the same one.  No key is 0 or 0xffffffff
// but a NaN's.
__device__ __forceinline__ uint32_t float_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t double_key(double x) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void max_shared_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void min_shared_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void add_shared_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_cluster_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// All threads of the cluster's C CTAs (C = 1: of the CTA) meet.
__device__ __forceinline__ void meet(int C) {
    if (C > 1) cluster_sync();
    else __syncthreads();
}

struct TopkShared {
    alignas(16) uint32_t hist[2][kTopkBins];
    alignas(16) uint32_t range[4];   // this CTA's least and largest key of the window, its keys above it and in it
    uint32_t warp_sum[32];
    uint32_t found[3];               // bin, keys above it, keys in it
    uint32_t warp_count[32][4];
    alignas(16) uint32_t count[2][4];  // this CTA's counts of cluster_counts
    uint32_t n_few, few[kTopkFew];   // this CTA's keys of cluster_finish,
    uint32_t all[kTopkFew];          // the cluster's
};
constexpr size_t kTopkSharedBytes = (sizeof(TopkShared) + 15) / 16 * 16;
constexpr int kTopkCtas = 8;  // of a cluster, at most (a portable size)

// Four values of every CTA of the cluster, at the same place of its shared memory: lane r of
// each warp gets CTA r's (lanes from C on: zeros).
__device__ __forceinline__ uint4 gather4(const uint32_t (&mine)[4], int C, int lane) {
    if (C == 1) return lane == 0 ? *reinterpret_cast<const uint4 *>(mine) : make_uint4(0u, 0u, 0u, 0u);
    return lane < C ? ld_shared_cluster_v4(map_shared_rank(smem_u32(mine), lane)) : make_uint4(0u, 0u, 0u, 0u);
}

// The keys from lo to hi, `inside` of them in all, that hold the m-th largest of them.
struct Border {
    uint32_t lo, hi, inside, m;
};

// The m-th largest of the keys key(i), i in [0, n), of the cluster's C CTAs lies in `w`: narrowed until
// it is one value (lo = hi), or all keys in it are among the m largest (m = inside), or there are at most
// `few`.  Every thread of the cluster calls it; `sh` lies at the same offset of every CTA's shared
// memory, its hist[0] is zero and the cluster has met since; it meets again before sh.hist is used again.
template <int kThreads, typename F>
__device__ Border cluster_narrow(F key, int n, Border w, int C, TopkShared &sh, uint32_t few) {
    constexpr int kPer = kTopkBins / kThreads;  // bins of a thread
    static_assert(kPer >= 4 && kPer % 4 == 0, "bins");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int buf = 0;
    while (w.lo != w.hi && w.m != w.inside && w.inside > few) {
        const uint32_t span = w.hi - w.lo;
        const int shift = max(0, 32 - __clz(static_cast<int>(span)) - kTopkBits);
        constexpr int kBatch = 4;  // keys read together (the additions would hold the next ones up)
        for (int i0 = tid; i0 - lane < n; i0 += kBatch * kThreads) {  // (whole warps)
            uint32_t k[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) k[j] = i0 + j * kThreads < n ? key(i0 + j * kThreads) : 0u;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const bool in = i0 + j * kThreads < n && k[j] >= w.lo && k[j] <= w.hi;
                const uint32_t bin = (k[j] - w.lo) >> shift;
                // a warp's keys in one bin, as many equal ones are: one addition
                const uint32_t act = __ballot_sync(0xffffffffu, in);
                const uint32_t first = __shfl_sync(0xffffffffu, bin, act ? __ffs(act) - 1 : 0);
                const bool one = __all_sync(0xffffffffu, !in || bin == first);
                if (in && (!one || lane == __ffs(act) - 1))
                    atomicAdd(&sh.hist[buf][bin], one ? static_cast<uint32_t>(__popc(act)) : 1u);
            }
        }
        meet(C);
        // the cluster's counts of this thread's bins, the highest bins the first thread's
        uint32_t cnt[kPer], sum = 0;
        const int bin0 = kTopkBins - (tid + 1) * kPer;
#pragma unroll
        for (int j = 0; j < kPer; j += 4) {
            uint4 v = *reinterpret_cast<const uint4 *>(&sh.hist[buf][bin0 + j]);
            if (C > 1) {
                const uint32_t at = smem_u32(&sh.hist[buf][bin0 + j]), me = cluster_ctarank();
                uint4 u[kTopkCtas - 1];
#pragma unroll
                for (int r = 1; r < kTopkCtas; ++r)
                    u[r - 1] = r < C ? ld_shared_cluster_v4(map_shared_rank(at, (me + r) % C)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int r = 0; r < kTopkCtas - 1; ++r) v.x += u[r].x, v.y += u[r].y, v.z += u[r].z, v.w += u[r].w;
            }
            cnt[j] = v.x, cnt[j + 1] = v.y, cnt[j + 2] = v.z, cnt[j + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += cnt[j];
        uint32_t upto = sum;  // counts of this thread's bins and of those above
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) sh.warp_sum[warp] = upto;
        for (int i = tid; i < kTopkBins; i += kThreads) sh.hist[buf ^ 1][i] = 0;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0u);
        uint32_t above = upto - sum;
        if (above < w.m && w.m <= upto) {
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j) {
                if (above < w.m && w.m <= above + cnt[j]) sh.found[0] = bin0 + j, sh.found[1] = above, sh.found[2] = cnt[j];
                above += cnt[j];
            }
        }
        __syncthreads();
        w.lo += sh.found[0] << shift;
        w.hi = min(w.hi - w.lo, (1u << shift) - 1u) + w.lo;
        w.m -= sh.found[1], w.inside = sh.found[2];
        buf ^= 1;
    }
    return w;
}

// Which keys hold the m-th largest (1 <= m <= their number) of all: those in the window [low, high], where
// most lie, those above it or those below.  `least`, `most`, `n_in`: of the keys in the window, the
// least, the largest and their number, `n_above`: the number of those above it.
__device__ __forceinline__ Border border_of(uint32_t m, uint32_t low, uint32_t high, uint32_t least, uint32_t most,
                                            uint32_t n_in, uint32_t n_above) {
    if (m <= n_above) return Border{high + 1u, ~0u, n_above, m};
    if (m <= n_above + n_in) return Border{least, most, n_in, m - n_above};
    return Border{0u, low - 1u, ~0u, m - n_above - n_in};
}

// What a thread has seen of its keys: the least and the largest in a window, how many lie in it, how
// many above it.
struct Window {
    uint32_t lo = ~0u, hi = 0u, in = 0u, above = 0u;

    __device__ __forceinline__ void see(uint32_t k, uint32_t low, uint32_t high) {
        const bool inside = k >= low && k <= high;
        lo = inside ? min(lo, k) : lo;
        hi = inside ? max(hi, k) : hi;
        above += k > high, in += inside;
    }
};

// The border of the m largest among the keys of all the cluster's CTAs, narrowed; `seen`: what this
// thread has seen of them, by the window [low, high].  The CTA meets before this (sh.warp_count has been
// read), the cluster before `sh` is used again.
template <int kThreads, typename F>
__device__ Border cluster_threshold(F key, int n, Window seen, uint32_t m, uint32_t low, uint32_t high, int C, TopkShared &sh,
                                    uint32_t few) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t lo = __reduce_min_sync(0xffffffffu, seen.lo), hi = __reduce_max_sync(0xffffffffu, seen.hi);
    uint32_t n_above = __reduce_add_sync(0xffffffffu, seen.above), n_in = __reduce_add_sync(0xffffffffu, seen.in);
    if (lane == 0) {
        sh.warp_count[warp][0] = lo, sh.warp_count[warp][1] = hi;
        sh.warp_count[warp][2] = n_above, sh.warp_count[warp][3] = n_in;
    }
    for (int i = tid; i < kTopkBins; i += kThreads) sh.hist[0][i] = 0;
    if (tid == 0) sh.n_few = 0;
    __syncthreads();
    if (warp == 0) {
        const bool w = lane < kWarps;
        lo = __reduce_min_sync(0xffffffffu, w ? sh.warp_count[lane][0] : ~0u);
        hi = __reduce_max_sync(0xffffffffu, w ? sh.warp_count[lane][1] : 0u);
        n_above = __reduce_add_sync(0xffffffffu, w ? sh.warp_count[lane][2] : 0u);
        n_in = __reduce_add_sync(0xffffffffu, w ? sh.warp_count[lane][3] : 0u);
        if (lane == 0) sh.range[0] = lo, sh.range[1] = hi, sh.range[2] = n_above, sh.range[3] = n_in;
    }
    meet(C);
    const uint4 r = gather4(sh.range, C, lane);
    lo = __reduce_min_sync(0xffffffffu, lane < C ? r.x : ~0u), hi = __reduce_max_sync(0xffffffffu, r.y);
    n_above = __reduce_add_sync(0xffffffffu, r.z), n_in = __reduce_add_sync(0xffffffffu, r.w);
    return cluster_narrow<kThreads>(key, n, border_of(m, low, high, lo, hi, n_in, n_above), C, sh, few);
}

// The border of cluster_threshold(few = kTopkFew), narrowed to one value: the keys left are listed and
// ranked, in one pass and one meeting (a further pass or two of cluster_narrow, 1 to 3 us each, otherwise).
// Once per kernel; the cluster meets before a CTA leaves.
template <int kThreads, typename F>
__device__ Border cluster_finish(F key, int n, Border w, int C, TopkShared &sh) {
    static_assert(kThreads >= kTopkFew * kTopkCtas, "a thread per key of every CTA");
    if (w.lo == w.hi || w.m == w.inside) return w;
    const int tid = threadIdx.x;
    constexpr int kBatch = 4;
    for (int i0 = tid; i0 < n; i0 += kBatch * kThreads) {
        uint32_t k[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) k[j] = i0 + j * kThreads < n ? key(i0 + j * kThreads) : 0u;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (i0 + j * kThreads < n && k[j] >= w.lo && k[j] <= w.hi) sh.few[atomicAdd(&sh.n_few, 1u)] = k[j];
    }
    meet(C);
    const int r = tid / kTopkFew, i = tid % kTopkFew;
    uint32_t here = 0, at = 0;  // keys of CTA r, and of those before it
    if (C == 1) {
        if (r == 0) here = sh.n_few;
        if (r == 0 && i < here) sh.all[i] = sh.few[i];
    } else if (r < C) {
        uint32_t c[kTopkCtas];
#pragma unroll
        for (int q = 0; q < kTopkCtas; ++q) c[q] = q < C ? ld_shared_cluster_u32(map_shared_rank(smem_u32(&sh.n_few), q)) : 0u;
        const uint32_t k = ld_shared_cluster_u32(map_shared_rank(smem_u32(&sh.few[i]), r));
#pragma unroll
        for (int q = 0; q < kTopkCtas; ++q) here = q == r ? c[q] : here, at += q < r ? c[q] : 0u;
        if (i < here) sh.all[at + i] = k;
    }
    __syncthreads();
    if (tid < w.inside) {
        const uint32_t mine = sh.all[tid];
        uint32_t above = 0, even = 0;
        for (uint32_t j = 0; j < w.inside; ++j) above += sh.all[j] > mine, even += sh.all[j] == mine;
        if (above < w.m && w.m <= above + even) sh.found[0] = mine, sh.found[1] = above, sh.found[2] = even;
    }
    __syncthreads();
    return Border{sh.found[0], sh.found[0], sh.found[2], w.m - sh.found[1]};
}

// Sums of N counts over the cluster's CTAs: *total, and over the CTAs of lower rank and this CTA's
// lower warps: *before.  `v`: this thread's.  Every thread of the cluster calls it; `slot` alternates
// between calls that no other meeting of the cluster lies between.
template <int kThreads, int N>
__device__ void cluster_counts(const uint32_t (&v)[N], int C, TopkShared &sh, int slot, uint32_t (&before)[N],
                               uint32_t (&total)[N]) {
    static_assert(N <= 4, "counts");
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t mine[N];
#pragma unroll
    for (int i = 0; i < N; ++i) mine[i] = __reduce_add_sync(0xffffffffu, v[i]);
    __syncthreads();  // (the last call's warp_count has been read)
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) sh.warp_count[warp][i] = mine[i];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t s = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_count[lane][i] : 0u);
            if (lane == i) sh.count[slot][i] = s;
        }
    }
    meet(C);
    const int me = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const uint4 q = gather4(sh.count[slot], C, lane);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        total[i] = __reduce_add_sync(0xffffffffu, u[i]);
        before[i] = __reduce_add_sync(0xffffffffu, (lane < me ? u[i] : 0u) + (lane < warp ? sh.warp_count[lane][i] : 0u));
    }
}

}  // namespace pa
