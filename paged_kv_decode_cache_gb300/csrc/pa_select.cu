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

// A sequence's length and its first touched block; false where it has none.
__device__ __forceinline__ bool touched_blocks(const BoundsArgs &a, int b, bool report, int *len, int *first) {
    int L = a.lens[b], from = a.starts ? a.starts[b] : 0;
    const int most = a.max_blocks * a.block_size;
    bool bad = L < 0 || L > most || from < 0;
    L = min(max(L, 0), most);
    from = max(from, 0);
    if (L - from > a.max_new) bad = true, from = L - a.max_new;
    if (bad && report) set_status(a.status, PA_STATUS_BAD_SEQLEN);
    *len = L, *first = from / a.block_size;
    return from < L;
}

// The bounds of 16 bytes of channels over rows slice, slice + step, ... of `rows`, kBatch of them on
// their way together; at: row 0's.
template <int kBatch, bool F8>
__device__ __forceinline__ void range_of_rows(Range<F8> &r, const uint4 *at, int64_t stride, int slice, int step, int rows) {
    for (int i0 = slice; i0 < rows; i0 += kBatch * step) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {  // (past the last row: the batch's first one again)
            const int i = i0 + k * step;
            v[k] = load_once(at + (i < rows ? i : i0) * stride);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) r.take(v[k], i0 == slice && k == 0);
    }
}

// Few blocks (a decode step's): a CTA per block that has new tokens.  Thread (slice, chunk)
// goes through every `slices`-th row of its 16 bytes of channels; the slices meet in shared
// memory.  Bound by the chain length - block id - keys.
template <bool F8>
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_kernel(const BoundsArgs a) {
    __shared__ uint4 part[2][kBoundsThreads];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, tid = threadIdx.x, bs = a.block_size;
    int L, first;
    if (!touched_blocks(a, b, tid == 0 && blockIdx.x == 0, &L, &first)) return;
    const int j = first + static_cast<int>(blockIdx.x);
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
            range_of_rows<8>(r, keys + c, a.row_chunks, slice, a.slices, rows);
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

// Many blocks (whole prompts): a CTA per 4 of them, a thread for 16 bytes of channels of a block, all
// of its rows.  Bound by memory: every key of the touched blocks is read once (360 MB in 53 us, the
// rate of a plain copy; 8 rows of a thread on their way leave room for half the threads: 60 us).
constexpr int kBoundsSpan = 4;
template <bool F8>
__global__ void __launch_bounds__(kBoundsThreads) key_bounds_many_kernel(const BoundsArgs a) {
    __shared__ int32_t ids[kBoundsSpan];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, tid = threadIdx.x, bs = a.block_size;
    int L, first;
    if (!touched_blocks(a, b, tid == 0 && blockIdx.x == 0, &L, &first)) return;
    const int j0 = first + static_cast<int>(blockIdx.x) * kBoundsSpan;
    if (j0 * bs >= L) return;
    if (tid < kBoundsSpan) {
        int phys = -1;
        if (j0 + tid < a.max_blocks && (j0 + tid) * bs < L) {
            phys = a.tables[static_cast<int64_t>(b) * a.max_blocks + j0 + tid];
            if (phys < 0 || phys >= a.num_blocks) {
                set_status(a.status, PA_STATUS_BAD_BLOCK);
                phys = -1;
            }
        }
        ids[tid] = phys;
    }
    __syncthreads();
    for (int i = tid; i < kBoundsSpan * a.row_chunks; i += kBoundsThreads) {
        const int k = i / a.row_chunks, c = i % a.row_chunks, phys = ids[k];
        if (phys < 0) continue;
        Range<F8> r;
        const uint4 *keys = reinterpret_cast<const uint4 *>(a.keys) + static_cast<int64_t>(phys) * bs * a.row_chunks;
        range_of_rows<4>(r, keys + c, a.row_chunks, 0, 1, min(bs, L - (j0 + k) * bs));
        uint4 *out = reinterpret_cast<uint4 *>(a.bounds) + static_cast<int64_t>(phys) * a.row_chunks * 2;
        out += 2 * (c / a.head_chunks) * a.head_chunks + c % a.head_chunks;
        out[0] = Range<F8>::pack(r.lo), out[a.head_chunks] = Range<F8>::pack(r.hi);
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
    int32_t room;            // keys in shared memory: blocks of a row, at most
    int32_t B, sorted;       // sorted: the longest sequences' clusters first
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 8;              // portable cluster size
constexpr int kSelMaxBlocks = 40960;     // of a sequence: their keys in one CTA's shared memory
constexpr uint32_t kSelFew = 32;         // the search for the border ends with so many keys near it
constexpr int kSelSorted = 256;          // sequences that are put in order, at a time
constexpr int kSelBatch = 4;             // keys that a thread reads together
constexpr int kSelList = 256;            // blocks near the border that are scored again at once
constexpr uint32_t kForced = 0xffffffffu;   // keys above every finite score's: blocks that are always taken ...
constexpr uint32_t kEndless = 0xfffffffeu;  // ... and blocks (or queries) with an infinity or a NaN
constexpr uint32_t kFirstFinite = 0x00800000u, kPastFinite = 0xff800000u;
// Of the sum of a score's |terms|, the error that its fp32 sum on tensor cores may have: 4
// sums of at most 4 MMAs, each adding 16 exact products to the sum after aligning all 17 to
// the largest, which cuts off at most 2^-23 of it from each, and 3 additions: 4 * 17 * 2^-23 +
// 2^-22 < 2^-16.
constexpr float kScoreError = 1.52587890625e-05f;
constexpr float kScoreFloor = 1e-35f;  // what products and sums below fp32's normal range lose, at most

// The larger |values| of three pairs of 16-bit ones (bf16, or fp16 for FP8 pools); a NaN stays.
template <bool F8>
__device__ __forceinline__ uint32_t largest2(uint32_t m, uint32_t u, uint32_t v) {
    if constexpr (F8) {
        const __half2 a = __habs2(*reinterpret_cast<__half2 *>(&u)), b = __habs2(*reinterpret_cast<__half2 *>(&v));
        const __half2 r = __hmax2_nan(__hmax2_nan(*reinterpret_cast<__half2 *>(&m), a), b);
        return *reinterpret_cast<const uint32_t *>(&r);
    } else {
        const __nv_bfloat162 a = __habs2(*reinterpret_cast<__nv_bfloat162 *>(&u)), b = __habs2(*reinterpret_cast<__nv_bfloat162 *>(&v));
        const __nv_bfloat162 r = __hmax2_nan(__hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&m), a), b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
}

// The z-th of the sequences by length, the longest first (of kSelSorted of them at a time, in their
// order among equals), by the CTA.
__device__ __forceinline__ int sequence_by_length(const SelectArgs &a, int z) {
    __shared__ __align__(16) int32_t lens_s[kSelSorted];
    __shared__ int32_t found_s;
    const int tid = threadIdx.x, base = z / kSelSorted * kSelSorted, n = min(kSelSorted, a.B - base);
    const int mine = tid < n ? a.lens[base + tid] : INT32_MIN;
    lens_s[tid] = mine;
    __syncthreads();
    int rank = 0;
    for (int j = 0; j < n; j += 4) {  // (those behind the last one are the least)
        const int4 x = *reinterpret_cast<const int4 *>(lens_s + j);
        rank += (x.x > mine || (x.x == mine && j < tid)) + (x.y > mine || (x.y == mine && j + 1 < tid)) +
                (x.z > mine || (x.z == mine && j + 2 < tid)) + (x.w > mine || (x.w == mine && j + 3 < tid));
    }
    if (tid < n && rank == z - base) found_s = tid;
    __syncthreads();
    return base + found_s;
}

// a + b = s + e, exactly.
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
    s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// The score of block `phys` for KV head h by one warp, as an ordered key: a sum in two fp32
// halves (products of bf16 are exact in fp32; such a sum keeps 45 bits and more), or, with
// `wide`, in 64 bits, for products that fp32's range does not hold (fp64 runs at a 64th of
// the rate).
template <bool F8, int D>
__device__ uint64_t exact_score(const SelectArgs &a, const float *q, int phys, int h, bool wide, int lane) {
    constexpr int kPer = D / 32;  // channels of a lane
    const uint8_t *row = a.bounds + (static_cast<int64_t>(phys) * a.Hkv + h) * 2 * D * (F8 ? 1 : 2);
    float x[2][kPer];  // lo, hi
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            if constexpr (F8) {
                const float2 f = f16x2_values(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(row + s * D + lane * kPer + i)));
                x[s][i] = f.x, x[s][i + 1] = f.y;
            } else {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(row + 2 * (s * D + lane * kPer + i));
                x[s][i] = bf16lo(w), x[s][i + 1] = bf16hi(w);
            }
        }
    }
    if (wide) {
        double top = -INFINITY;
        for (int g = 0; g < a.G; ++g) {
            double t = 0.0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float f = q[g * D + lane * kPer + i];
                t += static_cast<double>(f) * static_cast<double>(f < 0.f ? x[0][i] : x[1][i]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            top = t > top ? t : top;
        }
        return double_key(top);
    }
    float top_s = -INFINITY, top_e = 0.f;
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) {
        float s = 0.f, e = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float f = q[g * D + lane * kPer + i];
            float r;
            two_sum(s, __fmul_rn(f, f < 0.f ? x[0][i] : x[1][i]), s, r);
            e = __fadd_rn(e, r);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
            float r;
            two_sum(s, s2, s, r);
            e = __fadd_rn(__fadd_rn(e, e2), r);
        }
        two_sum(s, e, s, e);
        if (s > top_s || (s == top_s && e > top_e)) top_s = s, top_e = e;
    }
    return double_key(static_cast<double>(top_s) + static_cast<double>(top_e));
}

// A cluster per (sequence, KV head), a range of its blocks per CTA.  Each warp scores 16
// blocks at a time from registers and stores the scores, as ordered keys, in the first
// CTA's shared memory; the other CTAs leave, and that one finds the K-th largest
// (pa_topk.cuh) and writes the list.  (A search by all eight meets once a pass, 0.7 us, and
// took 15 of 48 us for 1025 blocks.)  A sum in fp32 does not tell neighbours apart that
// differ by less than its error, so blocks that the border may lie among (a few) are
// scored again, exactly for all that matters.  Bound by memory where a context is long (the
// bounds are read once), by the chain of loads, meetings and passes where it is short: 2 rows of
// 1025 blocks take 10 to 11 us, 32 rows of 2048 (34 MB) 16.5, 128 ragged FP8 rows of up to 8192 (135 MB) 54
// to 58.
template <bool F8, int D>
__global__ void __launch_bounds__(kSelThreads, 2) blocks_select_kernel(const SelectArgs a) {
    constexpr int kRowBytes = 2 * D * (F8 ? 1 : 2);
    constexpr int kChunks = kRowBytes / 64;             // 16-byte chunks of a row that a lane holds
    constexpr int kVecs = kChunks * Chunk<F8>::kVecs;   // vectors of 8 channels
    extern __shared__ __align__(16) uint8_t sel_smem[];
    TopkShared &sh = *reinterpret_cast<TopkShared *>(sel_smem);
    const int tiles = (a.G + 7) / 8;                    // of 8 query heads
    uint4 *qs = reinterpret_cast<uint4 *>(sel_smem + kTopkSharedBytes);   // [tiles][kVecs][32 lanes]: the MMA's columns
    float *qf = reinterpret_cast<float *>(qs + tiles * kVecs * 32);       // [G][D]
    uint32_t *keys = reinterpret_cast<uint32_t *>(qf + a.G * D);          // [room], the first CTA's
    __shared__ uint64_t wide_s[kSelList];       // blocks near the border: their exact scores as ordered keys,
    __shared__ int32_t list_s[kSelList];        // which they are
    __shared__ uint32_t window_s[4], largest_s; // the first CTA's: finite keys' least, largest, number; marks; largest bound
    __shared__ float qsum_s[32], qmax_s[32];    // sum of |q| of every head, -1 where one is not finite; the largest
    __shared__ uint32_t n_near_s, n_in_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int C = a.ctas, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int h = blockIdx.y, bs = a.block_size;
    griddep_wait();
    griddep_launch_dependents();
    const int b = a.sorted ? sequence_by_length(a, blockIdx.z) : static_cast<int>(blockIdx.z);

    // the queries' values, on their way with the length
    const int64_t row = static_cast<int64_t>(b) * a.Hkv + h;
    const uint32_t *q2 = reinterpret_cast<const uint32_t *>(a.q + row * a.G * D);
    for (int i = tid; i < a.G * D / 2; i += kSelThreads) {
        const uint32_t w = q2[i];
        *reinterpret_cast<float2 *>(qf + 2 * i) = make_float2(bf16lo(w), bf16hi(w));
    }
    int L = a.lens[b];
    const int most = a.max_blocks * bs;
    if (L < 0 || L > most) {
        if (tid == 0 && rank == 0 && h == 0) set_status(a.status, PA_STATUS_BAD_SEQLEN);
        L = L < 0 ? 0 : most;
    }
    const int n = (L + bs - 1) / bs;  // blocks
    const int32_t *bt = a.tables + static_cast<int64_t>(b) * a.max_blocks;
    int32_t *out = a.sel_tables + row * a.K;
    if (tid == 0 && rank == 0) a.sel_lens[row] = n <= a.K ? L : (a.K - 1) * bs + L - (n - 1) * bs;
    if (n <= a.K) {  // all of them
        for (int j = rank * kSelThreads + tid; j < a.K; j += C * kSelThreads) {
            const int id = j < n ? bt[j] : -1;
            if (j < n && (id < 0 || id >= a.num_blocks) && h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
            out[j] = id;
        }
        return;
    }
    if (tid == 0) window_s[0] = ~0u, window_s[1] = window_s[2] = window_s[3] = largest_s = 0u, n_near_s = n_in_s = 0u;
    for (int i = tid; i < kTopkBins; i += kSelThreads) sh.hist[0][i] = 0;
    if (C > 1) cluster_arrive();  // (every CTA has started and set these up before any stores to another's)

    // ---- a warp's tiles of 16 blocks: ids a tile ahead, the first tile's bounds on their way
    const int per = ((n + C - 1) / C + 15) / 16 * 16;
    const int j0 = min(rank * per, n), j1 = min(j0 + per, n);
    const int n_tiles = (j1 - j0 + 15) / 16;
    int next_id = lane < 16 && j0 + warp * 16 + lane < j1 ? bt[j0 + warp * 16 + lane] : -1;
    uint4 raw[2][kChunks];               // rows g and g + 8 of the tile on its way
    uint32_t ok;                         // its rows that are there
    auto load = [&](int tile, uint4(&k)[2][kChunks], uint32_t &there_all) {
        const int id = next_id, j = j0 + tile * 16 + (lane & 15);
        const bool fits = id >= 0 && id < a.num_blocks, here = lane < 16 && j < j1;
        if (here && !fits && h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
        there_all = __ballot_sync(0xffffffffu, here && fits);
        const int jn = j + kSelWarps * 16;
        next_id = lane < 16 && jn < j1 ? bt[jn] : -1;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int phys = __shfl_sync(0xffffffffu, id, g + 8 * r);
            const bool there = (there_all >> (g + 8 * r)) & 1u;
            const uint8_t *at = a.bounds + (static_cast<int64_t>(there ? phys : 0) * a.Hkv + h) * kRowBytes + 16 * t;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) k[r][c] = there ? load_once(at + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(warp, raw, ok);

    // ---- the sums of the queries' |values|, and the MMA's columns
    __syncthreads();
    for (int head = warp; head < a.G; head += kSelWarps) {
        float s = 0.f, m = 0.f;
        bool fine = true;
#pragma unroll
        for (int i = lane; i < D; i += 32) {
            const float x = fabsf(qf[head * D + i]);
            fine = fine && x < INFINITY;
            s += x, m = fmaxf(m, x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        fine = __all_sync(0xffffffffu, fine);
        if (lane == 0) qsum_s[head] = fine ? s : -1.f, qmax_s[head] = m;
    }
    __syncthreads();
    float qsum = 0.f, qmax = 0.f;
    bool q_fine = true;
    for (int i = 0; i < a.G; ++i) {
        q_fine = q_fine && qsum_s[i] >= 0.f;
        qsum = fmaxf(qsum, qsum_s[i]), qmax = fmaxf(qmax, qmax_s[i]);
    }
    // FP8: the columns are fp16, the queries scaled by a power of two so that the largest is below
    // 2^15 and not below 2^14; what that cuts off small ones is below 2^-39 of the largest
    const int shift = F8 && qmax > 0.f && q_fine ? 14 - ilogbf(qmax) : 0;
    const float up0 = exp2f(static_cast<float>(shift / 2)), up1 = exp2f(static_cast<float>(shift - shift / 2));
    const float down0 = 1.f / up0, down1 = 1.f / up1;  // (2^shift itself may lie outside fp32)
    for (int i = tid; i < tiles * kVecs * 32; i += kSelThreads) {
        const int ln = i & 31, v = (i >> 5) % kVecs, head = (i >> 5) / kVecs * 8 + (ln >> 2);
        const int x = vec_dim<F8>(v, ln & 3);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (head < a.G) {
            const float *f = qf + head * D + x % D;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float u = x >= D ? fmaxf(f[2 * k], 0.f) : fminf(f[2 * k], 0.f);
                const float y = x >= D ? fmaxf(f[2 * k + 1], 0.f) : fminf(f[2 * k + 1], 0.f);
                if constexpr (F8) {
                    w[k] = to_f16x2(u * up0 * up1, y * up0 * up1);
                } else {  // (the values are bf16)
                    w[k] = __float_as_uint(u) >> 16 | (__float_as_uint(y) & 0xffff0000u);
                }
            }
        }
        qs[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (C > 1) cluster_wait();
    __syncthreads();
    auto first = [&](void *p) { return C > 1 ? map_shared_rank(smem_u32(p), 0) : smem_u32(p); };  // in the first CTA
    const uint32_t keys0 = first(keys);

    // ---- scores
    uint32_t largest = 0u, w_lo = ~0u, w_hi = 0u, w_in = 0u, w_above = 0u;
    for (int tile = warp; tile < n_tiles; tile += kSelWarps) {
        uint32_t top[2] = {0u, 0u};  // largest |bound| of the rows, two of them side by side; a NaN stays
        float best[2] = {-INFINITY, -INFINITY};
        for (int nt = 0; nt < tiles; ++nt) {
            float part[4][4] = {}, acc[4];  // (four sums: shorter chains, and a quarter of the error)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                uint4 x[Chunk<F8>::kVecs], y[Chunk<F8>::kVecs];
                widen<F8>(raw[0][c], x);
                widen<F8>(raw[1][c], y);
#pragma unroll
                for (int k = 0; k < Chunk<F8>::kVecs; ++k) {
                    const int v = c * Chunk<F8>::kVecs + k;
                    const uint4 w = qs[(nt * kVecs + v) * 32 + lane];
                    mma_16x8x16<F8>(part[2 * v & 3], x[k].x, y[k].x, x[k].y, y[k].y, w.x, w.y);
                    mma_16x8x16<F8>(part[(2 * v + 1) & 3], x[k].z, y[k].z, x[k].w, y[k].w, w.z, w.w);
                    if (nt == 0) {
                        top[0] = largest2<F8>(largest2<F8>(top[0], x[k].x, x[k].y), x[k].z, x[k].w);
                        top[1] = largest2<F8>(largest2<F8>(top[1], y[k].x, y[k].y), y[k].z, y[k].w);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (nt * 8 + 2 * t + i < a.G) {
                    // (an overflow of finite values leaves the error infinite: any finite number will do)
                    const float u = F8 ? acc[i] * down0 * down1 : acc[i], v = F8 ? acc[2 + i] * down0 * down1 : acc[2 + i];
                    best[0] = fmaxf(best[0], u == u ? u : 0.f), best[1] = fmaxf(best[1], v == v ? v : 0.f);
                }
            }
        }
        const uint32_t there = ok;
        load(tile + kSelWarps, raw, ok);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float s = best[r];
            uint32_t m = top[r];
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
                m = largest2<F8>(m, __shfl_xor_sync(0xffffffffu, m, o), 0u);
            }
            const float2 mm = F8 ? f16x2_values(m) : make_float2(bf16lo(m), bf16hi(m));
            const bool fine = q_fine && mm.x < INFINITY && mm.y < INFINITY;
            const int j = j0 + tile * 16 + g + 8 * r;
            if (t == 0 && j < j1) {
                uint32_t key;
                if (j < a.first || j >= n - a.last) key = kForced;
                else if (!((there >> (g + 8 * r)) & 1u)) key = 0u;
                else if (!fine) key = kEndless;
                else key = float_key(fminf(fmaxf(s, -3.402823466e38f), 3.402823466e38f));
                if (C > 1) st_shared_cluster_u32(keys0 + 4 * j, key);
                else keys[j] = key;
                if (key >= kPastFinite) {
                    ++w_above;
                } else if (key) {
                    ++w_in, w_lo = min(w_lo, key), w_hi = max(w_hi, key);
                    largest = max(largest, __float_as_uint(fmaxf(mm.x, mm.y)));
                }
            }
        }
    }
    largest = __reduce_max_sync(0xffffffffu, largest);
    w_lo = __reduce_min_sync(0xffffffffu, w_lo), w_hi = __reduce_max_sync(0xffffffffu, w_hi);
    w_in = __reduce_add_sync(0xffffffffu, w_in), w_above = __reduce_add_sync(0xffffffffu, w_above);
    if (lane == 0) {
        const uint32_t w0 = first(window_s);
        min_shared_cluster_u32(w0, w_lo), max_shared_cluster_u32(w0 + 4, w_hi);
        add_shared_cluster_u32(w0 + 8, w_in), add_shared_cluster_u32(w0 + 12, w_above);
        max_shared_cluster_u32(first(&largest_s), largest);
    }
    if (C > 1) {
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
    }
    __syncthreads();

    // ---- the border, by the first CTA: taken are the keys above `to` and, of those from `from` to `to`, the first `need`
    largest = largest_s;
    auto key_at = [&](int i) { return keys[i]; };
    Border w = border_of(a.K, kFirstFinite, kPastFinite - 1u, window_s[0], window_s[1], window_s[2], window_s[3]);
    // (among the marks, and where every finite score is 0, keys are exact)
    const bool plain = w.lo >= kPastFinite || w.hi < kFirstFinite || !(qsum > 0.f && largest != 0u);
    w = cluster_narrow<kSelThreads>(key_at, n, w, 1, sh, plain ? 0u : kSelFew);
    uint32_t from = w.lo, to = w.hi, need = w.m == w.inside ? ~0u : w.m;
    if (!plain) {
        // every score is within err of its exact one, and so is the border: what is more than
        // 2 err from where the border may be is decided
        const float size = qsum * __uint_as_float(largest), err = fmaxf(kScoreError * size, kScoreFloor);
        const bool wide = !(size < 1e30f && size > 1e-18f);
        if (need == ~0u) to = from;  // (all from there on are the K largest: the border is at the least of them)
        uint32_t n_near, n_in;
        for (;;) {
            const uint32_t low = max(float_key(__fadd_rd(key_float(from), -2.f * err)), kFirstFinite);
            const uint32_t high = min(float_key(__fadd_ru(key_float(to), 2.f * err)), kPastFinite - 1u);
            uint32_t in = 0;
            for (int i0 = tid; i0 < n; i0 += kSelBatch * kSelThreads) {
                uint32_t k[kSelBatch];
#pragma unroll
                for (int j = 0; j < kSelBatch; ++j) k[j] = i0 + j * kSelThreads < n ? keys[i0 + j * kSelThreads] : 0u;
#pragma unroll
                for (int j = 0; j < kSelBatch; ++j) {
                    in += k[j] > high;
                    if (k[j] >= low && k[j] <= high) {
                        const uint32_t p = atomicAdd(&n_near_s, 1u);
                        if (p < kSelList) list_s[p] = i0 + j * kSelThreads;
                    }
                }
            }
            __syncwarp();
            in = __reduce_add_sync(0xffffffffu, in);
            if (lane == 0 && in) atomicAdd(&n_in_s, in);
            __syncthreads();
            n_near = n_near_s, n_in = n_in_s;
            if (from == to || n_near <= kSelList || n_near + n_in == a.K) {
                from = low, to = high;
                break;
            }
            for (int i = tid; i < kTopkBins; i += kSelThreads) sh.hist[0][i] = 0;
            __syncthreads();
            if (tid == 0) n_near_s = n_in_s = 0u;
            w = cluster_narrow<kSelThreads>(key_at, n, w, 1, sh, 0u);
            from = to = w.lo;  // (the K-th largest key, or a bound of those that are all taken)
            __syncthreads();
        }
        need = a.K - n_in;
        if (n_near == need) {
            need = ~0u;  // all of them
        } else if (n_near <= kSelList) {  // a warp per block, then ranked
            for (uint32_t p = warp; p < n_near; p += kSelWarps) {
                const uint64_t s = exact_score<F8, D>(a, qf, bt[list_s[p]], h, wide, lane);
                if (lane == 0) wide_s[p] = s;
            }
            __syncthreads();
            for (uint32_t p = tid; p < n_near; p += kSelThreads) {
                uint32_t better = 0;
                for (uint32_t o = 0; o < n_near; ++o)
                    better += wide_s[o] > wide_s[p] || (wide_s[o] == wide_s[p] && list_s[o] < list_s[p]);
                keys[list_s[p]] = better < need ? kForced : 0u;
            }
            need = 0u;
            __syncthreads();
        } else {
            // too many (hundreds of blocks that are nearly alike): 31 bits of their exact scores at a time, all
            // of them scored again for each (one row of 8192 blocks that are all alike: 3 ms, 32 such rows 4.6,
            // where bounds that differ take 42 us)
            const uint64_t last = double_key(static_cast<double>(key_float(to)) + 2.0 * err);
            uint64_t base = double_key(static_cast<double>(key_float(from)) - 2.0 * err);
            uint64_t span = last - base;
            for (;;) {
                const int shift = max(0, 64 - __clzll(static_cast<long long>(span)) - 31);
                Window seen;
                for (int i0 = warp * 32; i0 < n; i0 += kSelThreads) {
                    const int i = i0 + lane;
                    const uint32_t k = i < n ? keys[i] : 0u;
                    uint32_t now = k > to ? kForced : 0u;
                    for (uint32_t near = __ballot_sync(0xffffffffu, i < n && k >= from && k <= to); near; near &= near - 1) {
                        const int j = __ffs(near) - 1;
                        const uint64_t s = exact_score<F8, D>(a, qf, bt[i0 + j], h, wide, lane);
                        const uint64_t off = s < base ? 0u : min(s - base, span);
                        if (lane == j) now = static_cast<uint32_t>(off >> shift) + 1u;
                    }
                    if (i < n) keys[i] = now, seen.see(now, 1u, kForced - 1u);
                }
                __syncthreads();
                w = cluster_threshold<kSelThreads>(key_at, n, seen, a.K, 1u, kForced - 1u, 1, sh, 0u);
                from = w.lo, to = w.hi, need = w.m == w.inside ? ~0u : w.m;
                if (need == ~0u || shift == 0) break;
                base += static_cast<uint64_t>(from - 1u) << shift;
                span = (uint64_t(1) << shift) - 1u;
                __syncthreads();
            }
        }
    }

    // ---- the chosen blocks in their order: every warp's share of the row is contiguous
    const int share = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int i0 = min(warp * share, n), i1 = min(i0 + share, n);
    uint32_t taken[2] = {0, 0}, before[2], total[2];
    for (int i = i0 + lane; i < i1; i += 32) taken[0] += keys[i] > to, taken[1] += keys[i] >= from && keys[i] <= to;
    __syncwarp();
    cluster_counts<kSelThreads>(taken, 1, sh, 1, before, total);
    for (int i = i0; i < i1; i += 32 * kSelBatch) {
        uint32_t k[kSelBatch];
        int32_t id[kSelBatch];
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j) {  // (ids on their way together)
            const int x = i + 32 * j + lane;
            k[j] = x < i1 ? keys[x] : 0u;
            if (x < i1 && k[j] >= from) id[j] = bt[x];
        }
#pragma unroll
        for (int j = 0; j < kSelBatch; ++j) {
            const bool here = i + 32 * j + lane < i1, in = here && k[j] > to, even = here && k[j] >= from && k[j] <= to;
            const uint32_t ins = __ballot_sync(0xffffffffu, in), evens = __ballot_sync(0xffffffffu, even);
            const uint32_t below = (1u << lane) - 1u;
            const uint32_t tied = before[1] + __popc(evens & below);
            if (in || (even && tied < need)) out[before[0] + __popc(ins & below) + min(tied, need)] = id[j];
            before[0] += __popc(ins), before[1] += __popc(evens);
        }
    }
}

int bounds_slices(int row_chunks, int block_size) {
    int s = 1;
    while (s * 2 <= block_size && s * 2 * row_chunks <= kBoundsThreads && s < 32) s *= 2;
    return s;
}

size_t select_smem(int D, int G, int room) {
    return kTopkSharedBytes + static_cast<size_t>((G + 7) / 8) * (2 * D / 32) * 32 * 16 + static_cast<size_t>(G) * D * 4 +
           static_cast<size_t>(room) * 4;
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
                                 static_cast<int>(select_smem(D, 32, kSelMaxBlocks)));
        if (e != cudaSuccess) return e;
        smem_attr_done.fetch_or(bit, std::memory_order_release);
    }
    return launch_clustered(kern, dim3(a.ctas, a.Hkv, B), a.ctas, kSelThreads,
                            static_cast<int>(select_smem(D, a.G, a.room)), stream, pdl_on(), a);
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
    // The kernel for many blocks, where its CTAs fill the GPU several times over (16 prompts of 2048 to
    // 16384 tokens: 68 us with a CTA per block).
    const int sms = pa::sm_count();
    if (sms <= 0) return PA_ECUDA;
    const bool many = static_cast<int64_t>(blocks) * B >= 32ll * pa::kBoundsSpan * sms;
    auto kern = many ? (elem_bytes == 1 ? pa::key_bounds_many_kernel<true> : pa::key_bounds_many_kernel<false>)
                     : (elem_bytes == 1 ? pa::key_bounds_kernel<true> : pa::key_bounds_kernel<false>);
    const cudaError_t e = pa::launch_maybe_cooperative(
        kern, dim3(many ? (blocks + pa::kBoundsSpan - 1) / pa::kBoundsSpan : blocks, B), pa::kBoundsThreads, 0, stream, false,
        pa::pdl_on(), a);
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
    if (max_blocks_per_seq > pa::kSelMaxBlocks) return PA_EUNSUPPORTED;
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
    // a cluster of eight per row, or of fewer where those would run in more than two waves (128 rows of up
    // to 8192 blocks: 8 CTAs 60 us, 4 50, 2 80, 1 125)
    const int sms = pa::sm_count();
    if (sms <= 0) return PA_ECUDA;
    const int64_t rows = static_cast<int64_t>(B) * cache.num_kv_heads;
    a.ctas = pa::kSelCtas;
    while (a.ctas > 1 && rows * a.ctas > 4 * sms) a.ctas /= 2;
    a.room = max_blocks_per_seq;
    // the longest first where there is a second wave, which then has the short ones (62 -> 50 us; where
    // all run at once the order is 0.3 us of latency)
    a.B = B, a.sorted = B > 1 && rows * a.ctas > 2 * sms;
    cudaError_t e;
    if (elem_bytes == 1)
        e = cache.head_dim == 128 ? pa::launch_select<true, 128>(a, B, stream) : pa::launch_select<true, 64>(a, B, stream);
    else
        e = cache.head_dim == 128 ? pa::launch_select<false, 128>(a, B, stream) : pa::launch_select<false, 64>(a, B, stream);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // extern "C"
