// Selection of the m largest of many keys by the CTAs of a thread-block cluster, for
// pa_blocks_select and pa_cache_evict: a row's keys are spread over the cluster's
// shared memory, a contiguous range per CTA, and stay there.
//
// cluster_threshold finds the m-th largest key by narrowing a range of key values: each
// pass counts the keys of the range in 2048 equal bins (shared-memory atomics in every
// CTA, the counts added up through distributed shared memory) and keeps the bin that
// holds the border.  The range starts at the keys' own least and largest, so keys of
// one sign and a few exponents are split finely by the first pass; 32-bit keys take at
// most 3 passes, 64-bit ones 6.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kTopkBits = 11;
constexpr int kTopkBins = 1 << kTopkBits;

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
__device__ __forceinline__ uint64_t ld_shared_cluster_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
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
    alignas(16) uint64_t range[2];   // this CTA's least and largest key
    uint64_t warp_lo[32], warp_hi[32];
    uint32_t warp_sum[32];
    uint32_t found[3];               // bin, keys above it, keys in it
    uint32_t warp_count[32][4];
    alignas(16) uint32_t count[2][4];  // this CTA's counts of cluster_counts
};

// The m-th largest (1 <= m <= their number) of the keys key(i), i in [0, n), of the
// cluster's C CTAs; *need: how many of the keys equal to it are among the m largest.
// With `any`, a value between it and the next smaller key will do (and *need counts
// every key equal to it).  Every thread of the cluster calls it; `sh` lies at the same
// offset of every CTA's shared memory.  The caller meets the cluster before the CTAs'
// `sh` is used again or a CTA leaves.
template <typename Key, int kThreads, typename F>
__device__ Key cluster_threshold(F key, int n, uint32_t m, int C, TopkShared &sh, bool any, uint32_t *need) {
    constexpr int kWarps = kThreads / 32;
    constexpr int kPer = kTopkBins / kThreads;  // bins of a thread
    static_assert(kPer >= 4 && kPer % 4 == 0, "bins");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Key lo = ~Key(0), hi = 0;
    for (int i = tid; i < n; i += kThreads) {
        const Key k = key(i);
        lo = k < lo ? k : lo;
        hi = k > hi ? k : hi;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const Key a = __shfl_xor_sync(0xffffffffu, lo, d), b = __shfl_xor_sync(0xffffffffu, hi, d);
        lo = a < lo ? a : lo;
        hi = b > hi ? b : hi;
    }
    if (lane == 0) sh.warp_lo[warp] = lo, sh.warp_hi[warp] = hi;
    for (int i = tid; i < kTopkBins; i += kThreads) sh.hist[0][i] = 0;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) {
            lo = sh.warp_lo[w] < lo ? static_cast<Key>(sh.warp_lo[w]) : lo;
            hi = sh.warp_hi[w] > hi ? static_cast<Key>(sh.warp_hi[w]) : hi;
        }
        sh.range[0] = lo, sh.range[1] = hi;
    }
    meet(C);
    lo = static_cast<Key>(sh.range[0]), hi = static_cast<Key>(sh.range[1]);
    if (C > 1) {
        for (int r = 0; r < C; ++r) {
            const uint32_t at = map_shared_rank(smem_u32(sh.range), r);
            const Key a = static_cast<Key>(ld_shared_cluster_u64(at)), b = static_cast<Key>(ld_shared_cluster_u64(at + 8));
            lo = a < lo ? a : lo;
            hi = b > hi ? b : hi;
        }
    }
    int buf = 0;
    while (lo != hi) {
        const Key span = hi - lo;
        const int bits = sizeof(Key) == 8 ? 64 - __clzll(static_cast<long long>(span)) : 32 - __clz(static_cast<int>(span));
        const int shift = bits > kTopkBits ? bits - kTopkBits : 0;
        for (int i = tid; i - lane < n; i += kThreads) {  // (whole warps)
            const Key k = i < n ? key(i) : Key(0);
            const bool in = i < n && k >= lo && k <= hi;
            const uint32_t bin = static_cast<uint32_t>((k - lo) >> shift);
            // a warp's keys in one bin, as many equal ones are: one addition
            const uint32_t act = __ballot_sync(0xffffffffu, in);
            if (!act) continue;
            const uint32_t first = __shfl_sync(0xffffffffu, bin, __ffs(act) - 1);
            if (__all_sync(0xffffffffu, !in || bin == first)) {
                if (lane == 0) atomicAdd(&sh.hist[buf][first], static_cast<uint32_t>(__popc(act)));
            } else if (in) {
                atomicAdd(&sh.hist[buf][bin], 1u);
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
                for (int r = 1; r < C; ++r) {
                    const uint4 u = ld_shared_cluster_v4(map_shared_rank(at, (me + r) % C));
                    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
                }
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
        for (int w = 0; w < warp; ++w) upto += sh.warp_sum[w];
        uint32_t above = upto - sum;
        if (above < m && m <= upto) {
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j) {
                if (above < m && m <= above + cnt[j]) {
                    sh.found[0] = bin0 + j, sh.found[1] = above, sh.found[2] = cnt[j];
                }
                above += cnt[j];
            }
        }
        __syncthreads();
        const Key from = lo + (static_cast<Key>(sh.found[0]) << shift);
        const Key width = (Key(1) << shift) - 1;
        m -= sh.found[1];
        if (any && m == sh.found[2]) {  // the whole bin
            *need = ~0u;
            return from;
        }
        hi = hi - from < width ? hi : from + width;
        lo = from;
        buf ^= 1;
    }
    *need = m;
    return lo;
}

// Sums of N counts over the cluster's CTAs: *total, and over the CTAs of lower rank and this CTA's
// lower warps: *before.  `v`: this thread's.  Every thread of the cluster calls it; `slot` alternates
// between calls that no other meeting of the cluster lies between.
template <int kThreads, int N>
__device__ void cluster_counts(const uint32_t (&v)[N], int C, TopkShared &sh, int slot, uint32_t (&before)[N],
                               uint32_t (&total)[N]) {
    static_assert(N <= 4, "counts");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t mine[N];
#pragma unroll
    for (int i = 0; i < N; ++i) mine[i] = __reduce_add_sync(0xffffffffu, v[i]);
    __syncthreads();  // (the last call's warp_count has been read)
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) sh.warp_count[warp][i] = mine[i];
    __syncthreads();
    if (tid < N) {
        uint32_t s = 0;
        for (int w = 0; w < kThreads / 32; ++w) s += sh.warp_count[w][tid];
        sh.count[slot][tid] = s;
    }
    meet(C);
    const int me = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) before[i] = total[i] = 0;
    for (int r = 0; r < C; ++r) {
        const uint4 q = C > 1 ? ld_shared_cluster_v4(map_shared_rank(smem_u32(sh.count[slot]), r))
                              : *reinterpret_cast<const uint4 *>(sh.count[slot]);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (r < me) before[i] += u[i];
            total[i] += u[i];
        }
    }
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) before[i] += sh.warp_count[w][i];
}

}  // namespace pa
