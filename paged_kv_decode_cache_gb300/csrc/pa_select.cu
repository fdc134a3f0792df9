// Blocks chosen by a cheap score: every block's least and largest key per channel
// (pa_key_bounds), and the blocks whose bounds promise a query most (pa_blocks_select).
//
// For a key k of a block, lo <= k <= hi in every channel, so
//   q . k <= sum_d max(q_d lo_d, q_d hi_d) = [min(q, 0), max(q, 0)] . [lo, hi]:
// the score is a product with 2 D channels, which one MMA computes for 16 blocks and
// the query heads of a KV head (pa_mma.cuh).
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"
#include "pa_topk.cuh"

namespace pa {
namespace {

// ---- bounds ------------------------------------------------------------------------------

struct BoundsArgs {
    uint8_t *bounds;         // [num_blocks, Hkv, 2, D]
    const uint8_t *keys;     // [num_blocks, bs, Hkv, D]
    const int32_t *tables;   // [B, max_blocks]
    const int32_t *lens;     // [B]
    const int32_t *starts;   // [B] or null
    int32_t *status;
    int32_t num_blocks, block_size, max_blocks, max_new;
    int32_t row_chunks;      // 16-byte chunks of a token's keys
    int32_t head_chunks;     // of one head's
    int32_t slices;          // a block's rows are shared by so many threads
};

constexpr int kBoundsThreads = 256;

// Least and largest of 16 bytes' values each, NaN kept.
template <bool F8>
struct Range {
    static constexpr int kWords = F8 ? 8 : 4;  // two 16-bit values each: bf16, or fp16 for e4m3 codes
    uint32_t lo[kWords], hi[kWords];
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
        if constexpr (F8) {
            const __half2 r = __hmin2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&r);
        } else {
            const __nv_bfloat162 r =
                __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&r);
        }
    }
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
        if constexpr (F8) {
            const __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&r);
        } else {
            const __nv_bfloat162 r =
                __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&r);
        }
    }
    static __device__ __forceinline__ void words(const uint4 &v, uint32_t (&w)[kWords]) {
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (F8) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(in[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
                w[i] = static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
            } else {
                w[i] = in[i];
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const uint32_t (&w)[kWords]) {
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F8) {  // (exact: the values were codes)
                out[i] = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    __half2_raw h;
                    h.x = static_cast<unsigned short>(w[2 * i + k]), h.y = static_cast<unsigned short>(w[2 * i + k] >> 16);
                    out[i] |= static_cast<uint32_t>(__nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E4M3)) << (16 * k);
                }
            } else {
                out[i] = w[i];
            }
        }
        return make_uint4(out[0], out[1], out[2], out[3]);
    }
    __device__ __forceinline__ void take(const uint4 &v, bool first) {
        uint32_t w[kWords];
        words(v, w);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            lo[i] = first ? w[i] : least(lo[i], w[i]);
            hi[i] = first ? w[i] : most(hi[i], w[i]);
        }
    }
};

// A CTA per block that has new tokens.  Thread (slice, chunk) goes through every
// `slices`-th row of its 16 bytes of channels; the slices meet in shared memory.  Bound by
// memory: every key of the touched blocks is read once.
template <bool F8>
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_kernel(const BoundsArgs a) {
    __shared__ uint4 part[2][kBoundsThreads];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, tid = threadIdx.x, bs = a.block_size;
    int L = a.lens[b], from = a.starts ? a.starts[b] : 0;
    const int most = a.max_blocks * bs;
    bool bad = L < 0 || L > most || from < 0;
    L = min(max(L, 0), most);
    from = max(from, 0);
    if (L - from > a.max_new) bad = true, from = L - a.max_new;
    if (bad && tid == 0 && blockIdx.x == 0) set_status(a.status, PA_STATUS_BAD_SEQLEN);
    if (from >= L) return;
    const int j = from / bs + static_cast<int>(blockIdx.x);
    if (j * bs >= L) return;
    const int phys = a.tables[static_cast<int64_t>(b) * a.max_blocks + j];
    if (phys < 0 || phys >= a.num_blocks) {
        if (tid == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
        return;
    }
    const int rows = min(bs, L - j * bs);
    const uint4 *keys = reinterpret_cast<const uint4 *>(a.keys) + static_cast<int64_t>(phys) * bs * a.row_chunks;
    uint4 *out = reinterpret_cast<uint4 *>(a.bounds) + static_cast<int64_t>(phys) * a.row_chunks * 2;
    const int per = kBoundsThreads / a.slices;  // chunks of a turn
    const int slice = tid / per, lane = tid % per;
    for (int c0 = 0; c0 < a.row_chunks; c0 += per) {
        const int c = c0 + lane;
        const bool mine = slice < a.slices && c < a.row_chunks;
        if (mine && slice < rows) {
            Range<F8> r;
            const uint4 *at = keys + c;
            int i = slice;
            r.take(load_once(at + static_cast<int64_t>(i) * a.row_chunks), true);
            i += a.slices;
            for (; i + 3 * a.slices < rows; i += 4 * a.slices) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = load_once(at + static_cast<int64_t>(i + k * a.slices) * a.row_chunks);
#pragma unroll
                for (int k = 0; k < 4; ++k) r.take(v[k], false);
            }
            for (; i < rows; i += a.slices) r.take(load_once(at + static_cast<int64_t>(i) * a.row_chunks), false);
            part[0][tid] = Range<F8>::pack(r.lo), part[1][tid] = Range<F8>::pack(r.hi);
        }
        __syncthreads();
        if (mine && slice < 2) {  // slice 0 joins the least values, slice 1 the largest
            const int which0 = slice, which1 = a.slices == 1 ? 1 : slice;
            const int h = c / a.head_chunks, cc = c % a.head_chunks;
            for (int which = which0; which <= which1; ++which) {
                Range<F8> r;
                r.take(part[which][lane], true);
                for (int s = 1; s < min(a.slices, rows); ++s) r.take(part[which][s * per + lane], false);
                out[(2 * h + which) * a.head_chunks + cc] = Range<F8>::pack(which ? r.hi : r.lo);
            }
        }
        __syncthreads();
    }
}

// ---- selection ------------------------------------------------------------------------------

struct SelectArgs {
    int32_t *sel_tables;     // [B, Hkv, K]
    int32_t *sel_lens;       // [B, Hkv]
    const uint16_t *q;       // bf16 [B, Hq, D]
    const uint8_t *bounds;   // [num_blocks, Hkv, 2, D]
    const int32_t *tables;   // [B, max_blocks]
    const int32_t *lens;     // [B]
    int32_t *status;
    int32_t num_blocks, block_size, Hkv, G, max_blocks, K, first, last;
    int32_t ctas;            // of a cluster: a row of blocks
    int32_t slice;           // blocks of a CTA, at most
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 8;              // portable cluster size
constexpr int kSelMaxSlice = 12288;
constexpr uint32_t kForced = 0xffffffffu;   // keys above every finite score's: blocks that are always taken ...
constexpr uint32_t kEndless = 0xfffffffeu;  // ... and blocks (or queries) with an infinity or a NaN
constexpr uint32_t kFirstFinite = 0x00800000u, kPastFinite = 0xff800000u;
// Of the sum of a score's |terms|, the error that its fp32 sum on tensor cores may have: 16
// MMAs, each adding 16 exact products to the sum after aligning all 17 to the largest,
// which cuts off at most 2^-23 of it from each.  16 * 17 * 2^-23 < 2^-14.
constexpr float kScoreError = 6.103515625e-05f;
constexpr float kScoreFloor = 1e-35f;  // what products and sums below fp32's normal range lose, at most

// [min(q, 0), max(q, 0)] at channel x of 2 D.
__device__ __forceinline__ uint32_t signed_part(uint32_t q, bool upper) {
    return (q >> 15 != 0) != upper ? q : 0u;
}

// The score of block `phys` for KV head h in 64 bits, by one warp: the largest over the
// query heads, of which those that a sum in fp32 puts more than 2 * err below the best one
// are left out.
template <bool F8, int D>
__device__ double score64(const SelectArgs &a, const uint16_t *q, int phys, int h, float err, int lane) {
    constexpr int kPer = D / 32;
    const int d0 = lane * kPer;
    float lo[kPer], hi[kPer];
    const uint8_t *row = a.bounds + (static_cast<int64_t>(phys) * a.Hkv + h) * 2 * D * (F8 ? 1 : 2);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if constexpr (F8) {
            lo[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(row[d0 + i], __NV_E4M3)));
            hi[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(row[D + d0 + i], __NV_E4M3)));
        } else {
            const uint16_t *r = reinterpret_cast<const uint16_t *>(row);
            lo[i] = __uint_as_float(static_cast<uint32_t>(r[d0 + i]) << 16);
            hi[i] = __uint_as_float(static_cast<uint32_t>(r[D + d0 + i]) << 16);
        }
    }
    float best = -INFINITY;
    for (int pass = 0; pass < 2; ++pass) {
        double top = -INFINITY;
        for (int g = 0; g < a.G; ++g) {
            float f[kPer], s = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                f[i] = __uint_as_float(static_cast<uint32_t>(q[g * D + d0 + i]) << 16);
                s += fmaxf(f[i] * lo[i], f[i] * hi[i]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (pass == 0) {
                best = fmaxf(best, s);
            } else if (!(s < best - 2.f * err)) {  // (an overflow keeps every head)
                double t = 0.0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float x = f[i] < 0.f ? lo[i] : hi[i];
                    t += static_cast<double>(f[i]) * static_cast<double>(x);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                top = t > top ? t : top;
            }
        }
        if (pass == 1) return top;
    }
    return 0.0;
}

// A cluster per (sequence, KV head), a range of its blocks per CTA.  Each warp scores 16
// blocks at a time from registers; the scores stay in shared memory as ordered keys
// and the cluster finds the K-th largest (pa_topk.cuh).  A sum in fp32 does not tell
// neighbours apart that differ by less than its error, so blocks that the border may lie
// among (usually none or one) are scored again in 64 bits: what is chosen is what
// the 64-bit scores choose.  Bound by memory where a context is long (the bounds are read
// once), by the chain of loads, meetings and passes where it is short.
template <bool F8, int D>
__global__ void __launch_bounds__(kSelThreads, 2) blocks_select_kernel(const SelectArgs a) {
    constexpr int kRowBytes = 2 * D * (F8 ? 1 : 2);
    constexpr int kChunks = kRowBytes / 64;             // 16-byte chunks of a row that a lane holds
    constexpr int kVecs = kChunks * Chunk<F8>::kVecs;   // vectors of 8 channels
    extern __shared__ __align__(16) uint8_t sel_smem[];
    TopkShared &sh = *reinterpret_cast<TopkShared *>(sel_smem);
    const int tiles = (a.G + 7) / 8;                    // of 8 query heads
    uint4 *qs = reinterpret_cast<uint4 *>(sel_smem + (sizeof(TopkShared) + 15) / 16 * 16);  // [tiles][kVecs][32 lanes]
    uint64_t *wide = reinterpret_cast<uint64_t *>(qs + tiles * kVecs * 32);                 // [slice] 64-bit keys
    uint32_t *keys = reinterpret_cast<uint32_t *>(wide + a.slice);                          // [slice]
    uint16_t *list = reinterpret_cast<uint16_t *>(keys + a.slice);                          // [slice] whose they are
    __shared__ uint32_t largest_s;   // of the finite bounds, as a float's bits
    __shared__ float qsum_s[32];     // sum of |q| of every head, -1 where one is not finite
    __shared__ uint32_t n_wide_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int C = a.ctas, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int h = blockIdx.y, b = blockIdx.z, bs = a.block_size;
    griddep_wait();
    griddep_launch_dependents();

    int L = a.lens[b];
    const int most = a.max_blocks * bs;
    if (L < 0 || L > most) {
        if (tid == 0 && rank == 0 && h == 0) set_status(a.status, PA_STATUS_BAD_SEQLEN);
        L = L < 0 ? 0 : most;
    }
    const int n = (L + bs - 1) / bs;  // blocks
    const int32_t *bt = a.tables + static_cast<int64_t>(b) * a.max_blocks;
    const int64_t row = static_cast<int64_t>(b) * a.Hkv + h;
    int32_t *out = a.sel_tables + row * a.K;
    if (tid == 0 && rank == 0) a.sel_lens[row] = n <= a.K ? L : (a.K - 1) * bs + L - (n - 1) * bs;
    auto entry = [&](int j) {
        const int id = bt[j];
        const bool ok = id >= 0 && id < a.num_blocks;
        if (!ok && h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
        return id;
    };
    if (n <= a.K) {  // all of them
        for (int j = rank * kSelThreads + tid; j < a.K; j += C * kSelThreads) out[j] = j < n ? entry(j) : -1;
        return;
    }
    const int per = ((n + C - 1) / C + 15) / 16 * 16;
    const int j0 = min(rank * per, n), j1 = min(j0 + per, n), mine = j1 - j0;

    // ---- the queries as the MMA's columns, the sums of their |values|
    const uint16_t *q = a.q + row * a.G * D;
    for (int i = tid; i < tiles * kVecs * 32; i += kSelThreads) {
        const int ln = i & 31, v = (i >> 5) % kVecs, head = (i >> 5) / kVecs * 8 + (ln >> 2);
        const int x = vec_dim<F8>(v, ln & 3);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (head < a.G) {
            const uint4 in = *reinterpret_cast<const uint4 *>(q + head * D + x % D);
            const bool up = x >= D;
            auto both = [&](uint32_t u) { return signed_part(u & 0xffffu, up) | signed_part(u >> 16, up) << 16; };
            w = make_uint4(both(in.x), both(in.y), both(in.z), both(in.w));
        }
        qs[i] = w;
    }
    for (int head = warp; head < a.G; head += kSelWarps) {
        float s = 0.f;
        bool fine = true;
        for (int i = lane; i < D; i += 32) {
            const uint32_t u = q[head * D + i] & 0x7fffu;
            fine = fine && u < 0x7f80u;
            s += __uint_as_float(u << 16);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        fine = __all_sync(0xffffffffu, fine);
        if (lane == 0) qsum_s[head] = fine ? s : -1.f;
    }
    if (tid == 0) largest_s = 0u, n_wide_s = 0u;
    __syncthreads();
    float qsum = 0.f;
    bool q_fine = true;
    for (int i = 0; i < a.G; ++i) {
        q_fine = q_fine && qsum_s[i] >= 0.f;
        qsum = fmaxf(qsum, qsum_s[i]);
    }

    // ---- scores
    uint32_t largest = 0u;
    const int n_tiles = (mine + 15) / 16;
    int next = -1;
    if (warp < n_tiles && lane < 16 && j0 + warp * 16 + lane < j1) next = bt[j0 + warp * 16 + lane];
    for (int tile = warp; tile < n_tiles; tile += kSelWarps) {
        const int id = next, j_lane = j0 + tile * 16 + (lane & 15);
        const bool id_ok = lane < 16 && j_lane < j1 && id >= 0 && id < a.num_blocks;
        if (lane < 16 && j_lane < j1 && !id_ok && h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
        const uint32_t ok = __ballot_sync(0xffffffffu, id_ok);
        const int jn = j_lane + kSelWarps * 16;
        next = lane < 16 && jn < j1 ? bt[jn] : -1;
        uint4 raw[2][kChunks];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int phys = __shfl_sync(0xffffffffu, id, g + 8 * r);
            const bool there = (ok >> (g + 8 * r)) & 1u;
            const uint8_t *at = a.bounds + (static_cast<int64_t>(there ? phys : 0) * a.Hkv + h) * kRowBytes + 16 * t;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) raw[r][c] = there ? load_once(at + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t top[2] = {0u, 0u};  // largest |bound| of rows g and g + 8, per 16 (FP8: 8) bits
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t w[4] = {raw[r][c].x, raw[r][c].y, raw[r][c].z, raw[r][c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top[r] = F8 ? __vmaxu4(top[r], w[i] & 0x7f7f7f7fu) : __vmaxu2(top[r], w[i] & 0x7fff7fffu);
            }
        float best[2] = {-INFINITY, -INFINITY};
        for (int nt = 0; nt < tiles; ++nt) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                uint4 x[Chunk<F8>::kVecs], y[Chunk<F8>::kVecs];
                widen<F8>(raw[0][c], x);
                widen<F8>(raw[1][c], y);
#pragma unroll
                for (int k = 0; k < Chunk<F8>::kVecs; ++k) {
                    const uint4 w = qs[(nt * kVecs + c * Chunk<F8>::kVecs + k) * 32 + lane];
                    mma_16x8x16(acc, x[k].x, y[k].x, x[k].y, y[k].y, w.x, w.y);
                    mma_16x8x16(acc, x[k].z, y[k].z, x[k].w, y[k].w, w.z, w.w);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (nt * 8 + 2 * t + i < a.G) {
                    // (an overflow of finite values leaves the error infinite: any finite number will do)
                    const float u = acc[i], v = acc[2 + i];
                    best[0] = fmaxf(best[0], u == u ? u : 0.f), best[1] = fmaxf(best[1], v == v ? v : 0.f);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float s = best[r];
            uint32_t m = top[r];
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
                const uint32_t v = __shfl_xor_sync(0xffffffffu, m, o);
                m = F8 ? __vmaxu4(m, v) : __vmaxu2(m, v);
            }
            m = F8 ? max(max(m & 0xffu, (m >> 8) & 0xffu), max((m >> 16) & 0xffu, m >> 24)) : max(m & 0xffffu, m >> 16);
            const bool fine = q_fine && m < (F8 ? 0x7fu : 0x7f80u);
            const int i = tile * 16 + g + 8 * r, j = j0 + i;
            if (t == 0 && j < j1) {
                uint32_t key;
                if (j < a.first || j >= n - a.last) key = kForced;
                else if (!((ok >> (g + 8 * r)) & 1u)) key = 0u;
                else if (!fine) key = kEndless;
                else key = float_key(fminf(fmaxf(s, -3.402823466e38f), 3.402823466e38f));
                keys[i] = key;
                if (fine && key != kForced) {
                    const uint32_t f = F8 ? __float_as_uint(__half2float(__half(
                                                __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(m), __NV_E4M3))))
                                          : m << 16;
                    largest = max(largest, f);
                }
            }
        }
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
    if (lane == 0) atomicMax(&largest_s, largest);
    __syncthreads();

    // ---- the border
    const uint32_t m = a.K;
    uint32_t need;
    uint32_t border = cluster_threshold<uint32_t, kSelThreads>([&](int i) { return keys[i]; }, mine, m, C, sh, false, &need);
    uint32_t before[2], total[2];
    uint32_t past = border, tie = border;  // taken: keys above `past`, and the first `need` of those equal to `tie`
    if (border >= kFirstFinite && border < kPastFinite) {
        if (C > 1)
            for (int r = 0; r < C; ++r)
                largest = max(r ? largest : 0u, ld_shared_cluster_u32(map_shared_rank(smem_u32(&largest_s), r)));
        else
            largest = largest_s;
        // every score is within err of its 64-bit one, and so is the border: what is more than
        // 2 err from it is decided
        const float err = fmaxf(kScoreError * qsum * __uint_as_float(largest), kScoreFloor);
        if (qsum > 0.f && largest != 0u) {  // (else every score is 0, exactly)
            const float at = key_float(border);
            const uint32_t low = max(float_key(__fadd_rd(at, -2.f * err)), kFirstFinite);
            const uint32_t high = min(float_key(__fadd_ru(at, 2.f * err)), kPastFinite - 1u);
            uint32_t sides[2] = {0, 0};
            for (int i = tid; i < mine; i += kSelThreads) {
                const uint32_t k = keys[i];
                sides[0] += k > high, sides[1] += k >= low && k <= high;
            }
            cluster_counts<kSelThreads>(sides, C, sh, 0, before, total);
            if (total[1] == m - total[0]) {
                past = low - 1u, tie = 1u;  // (no key is 1)
            } else {
                // scored again, a warp per block
                for (int i0 = warp * 32; i0 < mine; i0 += kSelThreads) {
                    const uint32_t k = i0 + lane < mine ? keys[i0 + lane] : 0u;
                    uint32_t near = __ballot_sync(0xffffffffu, k >= low && k <= high);
                    for (; near; near &= near - 1) {
                        const int i = i0 + __ffs(near) - 1;
                        const double s = score64<F8, D>(a, q, bt[j0 + i], h, err, lane);
                        if (lane == 0) {
                            const uint32_t p = atomicAdd(&n_wide_s, 1u);
                            wide[p] = double_key(s), list[p] = static_cast<uint16_t>(i);
                        }
                    }
                }
                __syncthreads();
                const int n_wide = static_cast<int>(n_wide_s);
                const uint64_t edge = cluster_threshold<uint64_t, kSelThreads>([&](int p) { return wide[p]; }, n_wide,
                                                                               m - total[0], C, sh, false, &need);
                for (int p = tid; p < n_wide; p += kSelThreads)
                    keys[list[p]] = wide[p] > edge ? kForced : wide[p] == edge ? 1u : 0u;
                past = high, tie = 1u;
                __syncthreads();
            }
        }
    }

    // ---- the chosen blocks in their order: every warp's share of the range is contiguous
    const int share = ((mine + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int i0 = min(warp * share, mine), i1 = min(i0 + share, mine);
    uint32_t taken[2] = {0, 0};
    for (int i = i0 + lane; i < i1; i += 32) taken[0] += keys[i] > past, taken[1] += keys[i] <= past && keys[i] == tie;
    cluster_counts<kSelThreads>(taken, C, sh, 1, before, total);
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? keys[i + lane] : 0u;
        const bool in = i + lane < i1 && k > past, even = i + lane < i1 && !in && k == tie;
        const uint32_t ins = __ballot_sync(0xffffffffu, in), evens = __ballot_sync(0xffffffffu, even);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t tied = before[1] + __popc(evens & below);
        if (in || (even && tied < need)) out[before[0] + __popc(ins & below) + min(tied, need)] = bt[j0 + i + lane];
        before[0] += __popc(ins), before[1] += __popc(evens);
    }
    meet(C);  // (the others may still read this CTA's counts)
}

int bounds_slices(int row_chunks, int block_size) {
    int s = 1;
    while (s * 2 <= block_size && s * 2 * row_chunks <= kBoundsThreads && s < 32) s *= 2;
    return s;
}

size_t select_smem(bool f8, int D, int G, int slice) {
    return (sizeof(TopkShared) + 15) / 16 * 16 + static_cast<size_t>((G + 7) / 8) * (2 * D / 32) * 32 * 16 +
           static_cast<size_t>(slice) * 14;
}

template <bool F8, int D>
cudaError_t launch_select(SelectArgs &a, int B, cudaStream_t stream) {
    auto kern = blocks_select_kernel<F8, D>;
    static std::atomic<uint64_t> smem_attr_done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(smem_attr_done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(select_smem(F8, D, 32, kSelMaxSlice)));
        if (e != cudaSuccess) return e;
        smem_attr_done.fetch_or(bit, std::memory_order_release);
    }
    return launch_clustered(kern, dim3(a.ctas, a.Hkv, B), a.ctas, kSelThreads,
                            static_cast<int>(select_smem(F8, D, a.G, a.slice)), stream, pdl_on(), a);
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_key_bounds(void *bounds, const void *k_cache, int32_t elem_bytes, pa_cache_desc cache, const int32_t *block_tables,
                  int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *starts, int32_t max_new, int32_t B,
                  int32_t *status, pa_stream_t stream) {
    if (B < 0 || max_blocks_per_seq <= 0 || max_new < 0) return PA_EINVAL;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_EINVAL;
    const int rc = pa::check_cache(cache);
    if (rc) return rc;
    if (cache.num_kv_heads > 65535 || B > 65535) return PA_EUNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * cache.block_size > INT32_MAX / 2) return PA_EUNSUPPORTED;
    if (B == 0) return PA_OK;
    if (!bounds || !k_cache || !block_tables || !seq_lens) return PA_EINVAL;
    if (!pa::is_aligned(bounds, 16) || !pa::is_aligned(k_cache, 16) || !pa::is_aligned(block_tables, 4) ||
        !pa::is_aligned(seq_lens, 4) || !pa::is_aligned(starts, 4) || !pa::is_aligned(status, 4))
        return PA_EINVAL;
    const int32_t most = max_blocks_per_seq * cache.block_size;
    pa::BoundsArgs a{};
    a.bounds = static_cast<uint8_t *>(bounds), a.keys = static_cast<const uint8_t *>(k_cache);
    a.tables = block_tables, a.lens = seq_lens, a.starts = starts, a.status = status;
    a.num_blocks = cache.num_blocks, a.block_size = cache.block_size, a.max_blocks = max_blocks_per_seq;
    a.max_new = max_new == 0 ? most : std::min(max_new, most);
    a.head_chunks = cache.head_dim * elem_bytes / 16;
    a.row_chunks = a.head_chunks * cache.num_kv_heads;
    a.slices = pa::bounds_slices(a.row_chunks, cache.block_size);
    // so many new tokens lie in at most this many blocks
    const int blocks = std::min(max_blocks_per_seq, (a.max_new - 1 + cache.block_size - 1) / cache.block_size + 1);
    const cudaError_t e = pa::launch_maybe_cooperative(elem_bytes == 1 ? pa::key_bounds_kernel<true> : pa::key_bounds_kernel<false>,
                                                       dim3(blocks, B), pa::kBoundsThreads, 0, stream, false, pa::pdl_on(), a);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

int pa_blocks_select(int32_t *sel_tables, int32_t max_selected, int32_t *sel_lens, const void *q, const void *bounds,
                     int32_t elem_bytes, pa_cache_desc cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                     const int32_t *seq_lens, int32_t B, int32_t Hq, int32_t first, int32_t last, int32_t *status,
                     pa_stream_t stream) {
    if (B < 0 || max_blocks_per_seq <= 0 || max_selected <= 0 || first < 0 || last < 1) return PA_EINVAL;
    if (static_cast<int64_t>(first) + last > max_selected) return PA_EINVAL;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_EINVAL;
    const int rc = pa::check_cache(cache);
    if (rc) return rc;
    if (Hq <= 0 || Hq % cache.num_kv_heads != 0) return PA_EINVAL;
    if (Hq / cache.num_kv_heads > 32 || cache.num_kv_heads > 65535 || B > 65535) return PA_EUNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * cache.block_size > INT32_MAX / 2 ||
        static_cast<int64_t>(max_selected) * cache.block_size > INT32_MAX / 2)
        return PA_EUNSUPPORTED;
    if (max_blocks_per_seq > pa::kSelCtas * pa::kSelMaxSlice) return PA_EUNSUPPORTED;
    if (B == 0) return PA_OK;
    if (!sel_tables || !sel_lens || !q || !bounds || !block_tables || !seq_lens) return PA_EINVAL;
    if (!pa::is_aligned(q, 16) || !pa::is_aligned(bounds, 16) || !pa::is_aligned(sel_tables, 4) ||
        !pa::is_aligned(sel_lens, 4) || !pa::is_aligned(block_tables, 4) || !pa::is_aligned(seq_lens, 4) ||
        !pa::is_aligned(status, 4))
        return PA_EINVAL;
    pa::SelectArgs a{};
    a.sel_tables = sel_tables, a.sel_lens = sel_lens, a.q = static_cast<const uint16_t *>(q);
    a.bounds = static_cast<const uint8_t *>(bounds), a.tables = block_tables, a.lens = seq_lens, a.status = status;
    a.num_blocks = cache.num_blocks, a.block_size = cache.block_size, a.Hkv = cache.num_kv_heads;
    a.G = Hq / cache.num_kv_heads, a.max_blocks = max_blocks_per_seq, a.K = max_selected, a.first = first, a.last = last;
    a.ctas = pa::kSelCtas;
    a.slice = ((max_blocks_per_seq + a.ctas - 1) / a.ctas + 15) / 16 * 16;
    cudaError_t e;
    if (elem_bytes == 1)
        e = cache.head_dim == 128 ? pa::launch_select<true, 128>(a, B, stream) : pa::launch_select<true, 64>(a, B, stream);
    else
        e = cache.head_dim == 128 ? pa::launch_select<false, 128>(a, B, stream) : pa::launch_select<false, 64>(a, B, stream);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // extern "C"
