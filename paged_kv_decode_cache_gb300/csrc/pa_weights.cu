// The attention weight that cached tokens draw (pa_weights_add): for every sequence,
// KV head and token t
//   w[t] <- decay w[t] + sum over the queries i and the group's heads g that see t of
//           exp(scale <q_ig, K_t> - lse_ig),
// the softmax's own probabilities, rebuilt from the log-sum-exp that attention gave.  Every
// key is read once (by the tensor cores' kernel once per 256 columns).  A token's sum belongs to one
// warp, or, there, to two or four with a share of the columns each, whose sums another warp adds up in
// their order: no atomics, and the same bits every time.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

struct WeightsArgs {
    float *out;              // [B, Hkv, room]
    const float *old;        // the same, or out itself
    int32_t *positions;      // [B, Hkv, room] or null
    const uint16_t *q;       // bf16 [B, q_len, Hq, D]
    const float *lse;        // [B, q_len, Hq]
    const uint8_t *keys;     // [num_blocks, bs, Hkv, D]
    const int32_t *tables;   // [B, max_blocks]
    const int32_t *lens;     // [B]
    const int32_t *ends;     // [B] or null
    int32_t *status;
    int64_t room;
    int32_t num_blocks, block_size, Hkv, G, q_len, max_blocks;
    float scale_log2, decay;
};

constexpr int kWThreads = 256;
constexpr int kWWarps = kWThreads / 32;
constexpr int kWFew = 32;                               // columns (queries x heads) of the streaming kernel, at most

// The columns (query, head of the group) of a (sequence, KV head) into shared memory: the
// MMA's operands, the lse in log2 units, and the last token that each sees (-1: none).
template <bool F8, int D>
__device__ __forceinline__ void load_columns(const WeightsArgs &a, int b, int h, int first_new, int here, uint4 *qs,
                                             float *lse_s, int *last_s) {
    constexpr int kVecs = D / 32;
    const int tiles = (here + 7) / 8;
    for (int i = threadIdx.x; i < tiles * kVecs * 32; i += kWThreads) {
        const int ln = i & 31, v = (i >> 5) % kVecs, col = (i >> 5) / kVecs * 8 + (ln >> 2);
        const int64_t row = (static_cast<int64_t>(b) * a.q_len + col / a.G) * a.Hkv * a.G + h * a.G + col % a.G;
        uint4 w = col < here ? *reinterpret_cast<const uint4 *>(a.q + row * D + vec_dim<F8>(v, ln & 3))
                             : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (F8)
            w = make_uint4(to_f16x2(bf16lo(w.x), bf16hi(w.x)), to_f16x2(bf16lo(w.y), bf16hi(w.y)),
                           to_f16x2(bf16lo(w.z), bf16hi(w.z)), to_f16x2(bf16lo(w.w), bf16hi(w.w)));
        qs[i] = w;
    }
    for (int col = threadIdx.x; col < tiles * 8; col += kWThreads) {
        const int i = col / a.G;
        const int64_t row = (static_cast<int64_t>(b) * a.q_len + i) * a.Hkv * a.G + h * a.G + col % a.G;
        const float lse = col < here ? a.lse[row] : -INFINITY;
        lse_s[col] = lse * 1.4426950408889634f;
        last_s[col] = lse == -INFINITY ? -1 : first_new + i;  // (a query that saw nothing adds nothing)
    }
}

// What 8 columns add to the sums of rows g and g + 8 (tokens tok and tok + 8) of a tile.
__device__ __forceinline__ void add_columns(float (&sum)[2], const float (&acc)[4], float scale_log2, const float *lse,
                                            const int *last, int tok) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float z = lse[j];
        const int l = last[j];
        if (tok <= l) sum[0] += fast_exp2(fmaf(acc[j], scale_log2, -z));
        if (tok + 8 <= l) sum[1] += fast_exp2(fmaf(acc[2 + j], scale_log2, -z));
    }
}

// Up to 32 columns, as a decode step has: bound by the stream of keys.  A warp takes `pairs`
// pairs of 16-token tiles (32 tokens in a row), every eighth of its CTA's, and keeps 64
// registers of keys (8 KB a warp) on their way: a tile's registers are loaded again as soon
// as its products are done.  With up to 8 columns (kOne) the queries stay in registers.
// The four lanes that share a token add up two tiles at once and end with a token each, so
// that old and new weights are whole lines.  A 7B-shaped step (34 MB of keys) takes 7.7 us, 4 of
// them the launch and the first loads' chain; 32 ragged FP8 sequences of up to 16384 tokens (294
// MB) 58 to 68 us, 0.64 to 0.76 of a copy's rate.
template <bool F8, int D, bool kOne>
__global__ void __launch_bounds__(kWThreads, 2) weights_kernel(const WeightsArgs a, int pairs) {
    constexpr int kRowBytes = D * (F8 ? 1 : 2);
    constexpr int kChunks = kRowBytes / 64;
    constexpr int kV = Chunk<F8>::kVecs, kVecs = kChunks * kV;
    constexpr int kSlots = kChunks > 1 ? 8 / kChunks : 4;  // tiles on their way
    __shared__ uint4 qs[kWFew / 8 * kVecs * 32];           // [column tiles][kVecs][32 lanes]
    __shared__ float lse_s[kWFew];
    __shared__ int last_s[kWFew];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z, bs = a.block_size;
    griddep_wait();
    griddep_launch_dependents();
    int L = a.lens[b];
    const int most = static_cast<int>(min(static_cast<int64_t>(a.max_blocks) * bs, a.room));
    if (L < 0 || L > most) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) set_status(a.status, PA_STATUS_BAD_SEQLEN);
        L = L < 0 ? 0 : most;
    }
    constexpr int kPair = 2 * kTile, kStep = kWWarps * kPair;
    const int tok0 = static_cast<int>(blockIdx.x) * pairs * kStep;
    if (tok0 >= L) return;
    const int first_new = L - a.q_len;

    // the places of this warp's tiles in the pool, one per lane
    const int w0 = tok0 + warp * kPair;
    const int mine = min(pairs, w0 < L ? (L - w0 + kStep - 1) / kStep : 0);
    int place = -1;
    {
        const int at = w0 + (lane >> 1) * kStep + (lane & 1) * kTile;
        if ((lane >> 1) < mine && at < L) {
            const int phys = a.tables[static_cast<int64_t>(b) * a.max_blocks + at / bs];
            if (phys >= 0 && phys < a.num_blocks) place = phys * bs + at % bs;
            else if (h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
        }
    }
    const float *old = a.old + (static_cast<int64_t>(b) * a.Hkv + h) * a.room;
    float *out = a.out + (old - a.old);
    int32_t *positions = a.positions ? a.positions + (old - a.old) : nullptr;
    const uint8_t *keys = a.keys + h * kRowBytes + 16 * t;
    const int stride = a.Hkv * kRowBytes;                  // between rows
    uint4 raw[kSlots][2][kChunks];
    float was[kSlots / 2];
    auto load = [&](int i, uint4(&k)[2][kChunks]) {        // tile i
        const int at = __shfl_sync(0xffffffffu, place, i & 31);
        const int left = i < 2 * mine && at >= 0 ? L - (w0 + (i >> 1) * kStep + (i & 1) * kTile) - g : 0;
        const uint8_t *row = keys + static_cast<int64_t>(at + g) * stride;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                k[r][c] = left > 8 * r ? load_once(row + static_cast<int64_t>(8 * r) * stride + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
    };
    // of a pair's 32 tokens this lane ends with row g + 8 (t & 1) of tile t >> 1
    const int my_row = 16 * (t >> 1) + 8 * (t & 1) + g;
    auto load_old = [&](int p) {
        const int x = w0 + p * kStep + my_row;
        return p < mine && x < first_new ? old[x] : 0.f;
    };
#pragma unroll
    for (int s = 0; s < kSlots; ++s) load(s, raw[s]);
#pragma unroll
    for (int s = 0; s < kSlots / 2; ++s) was[s] = load_old(s);
    const int columns = a.q_len * a.G, col_tiles = kOne ? 1 : (columns + 7) / 8;
    load_columns<F8, D>(a, b, h, first_new, columns, qs, lse_s, last_s);
    __syncthreads();
    const int shift = a.ends ? a.ends[b] - L : 0;  // a token's position less its place
    uint4 q1[kOne ? kVecs : 1];
    float lse1[2];
    int last1[2];
    if constexpr (kOne) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) q1[v] = qs[v * 32 + lane];
#pragma unroll
        for (int j = 0; j < 2; ++j) lse1[j] = lse_s[2 * t + j], last1[j] = last_s[2 * t + j];
    }

    for (int p0 = 0; p0 < mine; p0 += kSlots / 2) {
#pragma unroll
        for (int ps = 0; ps < kSlots / 2; ++ps) {
            const int p = p0 + ps;
            if (p >= mine) break;
            float sum[2][2] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint4(&k)[2][kChunks] = raw[2 * ps + e];
                const int tok = w0 + p * kStep + e * kTile + g;
                for (int nt = 0; nt < col_tiles; ++nt) {
                    float acc[2][4] = {};  // (two sums: half the chain)
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        uint4 x[kV], y[kV];
                        widen<F8>(k[0][c], x);
                        widen<F8>(k[1][c], y);
#pragma unroll
                        for (int j = 0; j < kV; ++j) {
                            const uint4 w = kOne ? q1[kOne ? c * kV + j : 0] : qs[(nt * kVecs + c * kV + j) * 32 + lane];
                            mma_16x8x16<F8>(acc[0], x[j].x, y[j].x, x[j].y, y[j].y, w.x, w.y);
                            mma_16x8x16<F8>(acc[1], x[j].z, y[j].z, x[j].w, y[j].w, w.z, w.w);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[0][i] += acc[1][i];
                    if constexpr (kOne) add_columns(sum[e], acc[0], a.scale_log2, lse1, last1, tok);
                    else add_columns(sum[e], acc[0], a.scale_log2, lse_s + nt * 8 + 2 * t, last_s + nt * 8 + 2 * t, tok);
                }
                load(2 * (p + kSlots / 2) + e, k);
            }
            const float before = was[ps];
            was[ps] = load_old(p + kSlots / 2);
            // rows g and g + 8 of two tiles over four lanes: lane t keeps tile t >> 1, row 8 (t & 1)
            const float give0 = t & 1 ? sum[0][0] : sum[0][1], give1 = t & 1 ? sum[1][0] : sum[1][1];
            const float v0 = (t & 1 ? sum[0][1] : sum[0][0]) + __shfl_xor_sync(0xffffffffu, give0, 1);
            const float v1 = (t & 1 ? sum[1][1] : sum[1][0]) + __shfl_xor_sync(0xffffffffu, give1, 1);
            float v = (t & 2 ? v1 : v0) + __shfl_xor_sync(0xffffffffu, t & 2 ? v0 : v1, 2);
            const int at = __shfl_sync(0xffffffffu, place, (2 * p + (t >> 1)) & 31);
            const int x = w0 + p * kStep + my_row;
            if (x < L) {
                if (at < 0) v = 0.f;  // (a block outside the pool)
                const bool fresh = x >= first_new;
                out[x] = fresh ? v : fmaf(a.decay, before, v);
                if (fresh && positions) positions[x] = x + shift;
            }
        }
    }
}

// ---- more columns (a window of queries over a long context): tensor cores --------------------
//
// S[128 tokens, N] = K[128, D] . Q^T[D, N] per tile, N <= 256 columns (query, head of the group)
// at a time, by tcgen05.mma into one of two buffers in TMEM; groups of four warps, each with
// a share of the columns, add up their rows' exponentials, and the last warp joins the groups'
// sums and writes the weights.  Per tile N products of 128 x D (0.5 us for 224 columns), 128 N
// exponentials (0.5 us at 32 a clock) and 32 KB of keys (0.75 us at an SM's share of the
// memory), all overlapped.  -lse stays in registers, a thread's columns being the same in every
// row: loads of it from shared memory compete with the MMA's operands there.  32 queries of 7 heads
// over 4 x 32768 tokens take 38 us (memory alone: 20) on 144 of 152 SMs: 10 of start and end and
// 0.98 for each of a CTA's 29 tiles (8192 tokens, 8 tiles: 17.7; 16384, 15 tiles: 24.5); 6 queries 30:
// 7 and 0.8.
//
// Keys come into a ring of stages as the MMA reads them (K-major, 128-byte swizzle): by TMA from
// one warp (8 warps of asynchronous copies: 5 us more), or for FP8 pools by 8 warps, which widen the
// codes to fp16 on the way (54 us, 1.5 a tile: bound by that).  Every wait is bounded.
constexpr int kXColumns = 256;           // at once
template <bool F8>
struct XWarps {
    static constexpr int kGroups = F8 ? 2 : 4;       // of four warps, for the exponentials (F8: registers for no more)
    static constexpr int kPart = kXColumns / kGroups;  // columns of a group, at most
    static constexpr int kLoad = 4 * kGroups;        // the first loading warp, after the exponentials'
    static constexpr int kMma = kLoad + (F8 ? 8 : 1);
    static constexpr int kFinal = kMma + 1;
    static constexpr int kThreads = 32 * (kFinal + 1);
};
constexpr int kXLoadRows = 16;           // FP8: tokens of a loading warp
constexpr int kXRows = 128;              // tokens of a tile
constexpr int kXAhead = 2;               // FP8: tiles whose copies are on their way
constexpr int kXCodes = kXAhead + 1;     // FP8: tiles in the ring of codes
constexpr int kXLook = 4;                // tiles whose old weights are on their way
constexpr int kXMostTiles = 32;          // of a CTA

template <bool F8, int D>
struct XShape {
    static constexpr int kHalves = D / 64;                       // 64-element sub-rows
    static constexpr int kStages = F8 ? 2 : 4;
    static constexpr int kStageBytes = kHalves * kXRows * kSubBytes;
    // dynamic shared memory: stages, codes, queries, sums, -lse, last tokens, groups' sums, barriers, places
    static constexpr int kCodeBytes = F8 ? kXCodes * kXRows * D : 0;
    static constexpr int q_bytes(int n) { return kHalves * n * kSubBytes; }
    static constexpr int q_at() { return kStages * kStageBytes + kCodeBytes; }
    static constexpr int sums_at(int n) { return q_at() + q_bytes(n); }
    static constexpr int bytes(int n) {
        return sums_at(n) + kXMostTiles * kXRows * 4 + 2 * kXColumns * 4 + 4 * XWarps<F8>::kGroups * kXRows * 4 +
               (2 * kStages + 13) * 8 + 16 + kXMostTiles * kXRows / kTile * 4 + 1024;
    }
};

// The sums over the columns below n1 of a warp's 32 rows in TMEM of 2^(s scale + nl), nl of this
// thread's columns in registers.  Thread t reads columns 2 (t % 4), + 1 (mod 8) of rows t / 4 + 8 k; the
// four lanes of a row then add up, and thread t ends with row t / 4 + 8 (t % 4).  kMasked: only columns
// that see the row's token, tok + the row.
template <bool kMasked, int kCols>
__device__ __forceinline__ float row_sums(uint32_t rows, int n1, float scale, const uint64_t (&nl)[kCols / 8], const int *last,
                                          int tok) {
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    const uint64_t scale2 = pack2(scale, scale);
    uint64_t sum2[4] = {0u, 0u, 0u, 0u};  // two columns' sums side by side
    uint32_t x[2][16];                    // (one is on its way while the other is added up)
    auto add = [&](auto whole, int half, int blk) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 32 * blk + 8 * r + 2 * t;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float e0, e1;
                unpack2(fma2(pack2(__uint_as_float(x[half][4 * r + 2 * k]), __uint_as_float(x[half][4 * r + 2 * k + 1])), scale2,
                             nl[4 * blk + r]), e0, e1);
                e0 = fast_exp2(e0), e1 = fast_exp2(e1);
                if constexpr (!whole.value) {
                    const int seer = tok + g + 16 * half + 8 * k;
                    e0 = n < n1 && (!kMasked || seer <= last[n]) ? e0 : 0.f;
                    e1 = n + 1 < n1 && (!kMasked || seer <= last[n + 1]) ? e1 : 0.f;
                }
                sum2[2 * half + k] = add2(sum2[2 * half + k], pack2(e0, e1));
            }
        }
    };
    auto add_block = [&](auto whole, int blk) {
        tc5::wait_ld_of(x[0]);
        tc5::ld_16x256b_x4_nowait(rows + (16u << 16) + 32 * blk, x[1]);
        add(whole, 0, blk);
        tc5::wait_ld_of(x[1]);
        if (32 * blk + 32 < n1) tc5::ld_16x256b_x4_nowait(rows + 32 * blk + 32, x[0]);
        add(whole, 1, blk);
    };
    if (n1 > 0) tc5::ld_16x256b_x4_nowait(rows, x[0]);
#pragma unroll
    for (int blk = 0; blk < kCols / 32; ++blk) {
        if (32 * blk >= n1) break;
        if (!kMasked && 32 * blk + 32 <= n1) add_block(std::true_type{}, blk);
        else add_block(std::false_type{}, blk);
    }
    float sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float e0, e1;
        unpack2(sum2[k], e0, e1);
        sum[k] = e0 + e1;
    }
    const float v0 = (t & 1 ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, t & 1 ? sum[0] : sum[1], 1);
    const float v1 = (t & 1 ? sum[3] : sum[2]) + __shfl_xor_sync(0xffffffffu, t & 1 ? sum[2] : sum[3], 1);
    return (t & 2 ? v1 : v0) + __shfl_xor_sync(0xffffffffu, t & 2 ? v0 : v1, 2);
}

template <bool F8, int D>
__global__ void __launch_bounds__(XWarps<F8>::kThreads, 1)
weights_tc_kernel(const __grid_constant__ CUtensorMap map, const WeightsArgs a, int tiles_max, int n_most, uint32_t tmem_cols) {
    using X = XShape<F8, D>;
    constexpr int kXStages = X::kStages, kXThreads = XWarps<F8>::kThreads;
    constexpr int kXLoadWarp = XWarps<F8>::kLoad, kXMmaWarp = XWarps<F8>::kMma, kXFinalWarp = XWarps<F8>::kFinal;
    constexpr int kGroups = XWarps<F8>::kGroups;
    extern __shared__ uint8_t x_smem[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(x_smem) + 1023) & ~uintptr_t(1023));
    uint8_t *codes = smem + kXStages * X::kStageBytes, *qs = smem + X::q_at();
    float *sums = reinterpret_cast<float *>(smem + X::sums_at(n_most));      // [tiles][128], over the chunks of columns
    float *nl = sums + kXMostTiles * kXRows;                                  // -lse of every column, log2 units
    int *last_s = reinterpret_cast<int *>(nl + kXColumns);                    // last token that it sees
    float *other = reinterpret_cast<float *>(last_s + kXColumns);             // [4][groups][128]: a tile's sums by group
    uint64_t *bars = reinterpret_cast<uint64_t *>(other + 4 * kGroups * kXRows);
    uint64_t *kfull = bars, *kempty = bars + kXStages;              // a stage holds keys, has been read
    uint64_t *sdone = bars + 2 * kXStages, *sfree = sdone + 2;      // a buffer holds scores, has been read
    uint64_t *hdone = sfree + 2, *hfree = hdone + 4;                // a slot holds the groups' sums, has been read
    uint64_t *drain = hfree + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *places = reinterpret_cast<int *>(tmem_slot + 2);                     // of 16 tokens each, -1: none
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, b = blockIdx.z, bs = a.block_size;
    griddep_wait();
    griddep_launch_dependents();
    int L = a.lens[b];
    const int most = static_cast<int>(min(static_cast<int64_t>(a.max_blocks) * bs, a.room));
    if (L < 0 || L > most) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) set_status(a.status, PA_STATUS_BAD_SEQLEN);
        L = L < 0 ? 0 : most;
    }
    const int tok0 = static_cast<int>(blockIdx.x) * tiles_max * kXRows;
    if (tok0 >= L) return;
    const int tiles = min(tiles_max, (L - tok0 + kXRows - 1) / kXRows);
    const int first_new = L - a.q_len, n_cols = a.q_len * a.G;
    const int32_t *table = a.tables + static_cast<int64_t>(b) * a.max_blocks;

    if (warp == kXMmaWarp) tc5::tmem_alloc(tmem_slot, tmem_cols);
    if (tid == 0) {
        for (int i = 0; i < kXStages; ++i) mbar_init(&kfull[i], F8 ? 32 * (kXMmaWarp - kXLoadWarp) : 1), mbar_init(&kempty[i], 1u);
        for (int i = 0; i < 4; ++i) mbar_init(&hdone[i], 4u * kGroups), mbar_init(&hfree[i], 1u);
        for (int i = 0; i < 2; ++i) mbar_init(&sdone[i], 1u), mbar_init(&sfree[i], 4u * kGroups);
        mbar_init(drain, 1u);
        *abort_flag = 0;
    }
    fence_barrier_init();
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return mbar_try_wait(bar, parity) || mbar_wait_or_abort_slow(bar, parity, abort_flag, a.status);
    };

    const bool loads = warp >= kXLoadWarp && warp < kXMmaWarp;
    bool good = true;
    uint32_t tmem = 0;
    int it = 0;   // tiles of the chunks before this one
    for (int c0 = 0; c0 < n_cols; c0 += n_most, it += tiles) {
        const int here = min(n_most, n_cols - c0), N = (here + 15) / 16 * 16;
        const bool first = c0 == 0, final = c0 + here == n_cols;
        const int part = ((N + kGroups - 1) / kGroups + 31) / 32 * 32;  // a group's columns
        const uint32_t width = tmem_cols / 2;                           // tile u is in buffer u & 1
        // (the chunk before this one is read; TMEM and the barriers are set up)
        if (__syncthreads_or(!first && *abort_flag != 0)) break;
        tmem = *tmem_slot;
        for (int i = tid; i < N * (D / 8); i += kXThreads) {
            const int n = i / (D / 8), ch = i % (D / 8);
            const int64_t row = (static_cast<int64_t>(b) * a.q_len + (c0 + n) / a.G) * a.Hkv * a.G + h * a.G + (c0 + n) % a.G;
            uint4 w = n < here ? *reinterpret_cast<const uint4 *>(a.q + row * D + 8 * ch) : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (F8)
                w = make_uint4(to_f16x2(bf16lo(w.x), bf16hi(w.x)), to_f16x2(bf16lo(w.y), bf16hi(w.y)),
                               to_f16x2(bf16lo(w.z), bf16hi(w.z)), to_f16x2(bf16lo(w.w), bf16hi(w.w)));
            *reinterpret_cast<uint4 *>(qs + (ch >> 3) * (N * kSubBytes) + swz128(n, ch & 7)) = w;
        }
        // the places in the pool of all tiles' 16 tokens each, looked up at once
        if (first) {
            for (int x = tid; x < tiles * (kXRows / kTile); x += kXThreads) {
                const int tok = tok0 + x * kTile, phys = tok < L ? table[tok / bs] : -1;
                const bool fits = phys >= 0 && phys < a.num_blocks;
                if (tok < L && !fits && h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
                places[x] = fits ? phys * bs + tok % bs : -1;
            }
        }
        bool no_lse = false;
        for (int n = tid; n < N; n += kXThreads) {
            const int i = (c0 + n) / a.G;
            const int64_t row = (static_cast<int64_t>(b) * a.q_len + i) * a.Hkv * a.G + h * a.G + (c0 + n) % a.G;
            const float lse = n < here ? a.lse[row] : 0.f;
            nl[n] = -lse * 1.4426950408889634f;
            last_s[n] = lse == -INFINITY ? -1 : first_new + i;
            no_lse = no_lse || lse == -INFINITY;
        }
        fence_proxy_async_smem();
        tc5::fence_before_sync();
        const bool odd = __syncthreads_or(no_lse);  // a column of the chunk has no lse
        tc5::fence_after_sync();

        if (loads) {
            if constexpr (!F8) {
                // lane 2 i + half: 16 tokens of a tile, 64 channels.  (Places of no token, and tokens of a block
                // outside the pool, keep what the stage had: their rows' scores are not used.)
                const int sub = lane / X::kHalves, half = lane % X::kHalves;
                const bool carrier = sub < kXRows / kTile;
                const uint64_t policy = l2_evict_first_policy();
                int issued = it;
                for (int i = 0; i < tiles && good; ++i) {
                    const int u = it + i, s = u % kXStages, place = carrier ? places[i * (kXRows / kTile) + sub] : -1;
                    const bool valid = place >= 0;
                    const uint32_t copies = __popc(__ballot_sync(0xffffffffu, valid));
                    if (u >= kXStages) good = __all_sync(0xffffffffu, wait(&kempty[s], (u / kXStages - 1) & 1));
                    if (!good) break;
                    if (lane == 0) mbar_arrive_expect_tx(&kfull[s], copies * kTile * kSubBytes);
                    __syncwarp();
                    if (valid)
                        tma_load_4d(smem + s * X::kStageBytes + half * (kXRows * kSubBytes) + sub * kTile * kSubBytes, &map, 0,
                                    place, h, half, &kfull[s], policy);
                    issued = u + 1;
                }
                // (the copies land before this CTA leaves, whatever became of the other warps)
                for (int u = max(0, issued - kXStages); u < issued; ++u) mbar_wait_bounded(&kfull[u % kXStages], (u / kXStages) & 1);
            } else {
                // A loading warp's 16 rows of a tile: kPer chunks of 16 bytes a lane, copied
                // asynchronously kXAhead tiles ahead into the lane's own part of a ring of codes, which it
                // widens into the stage later.  The fence to the MMA's proxy is the MMA warp's, after the
                // stage's barrier: here it would wait for the copies of the next tiles, too.
                constexpr int kRowChunks = D / 16, kPer = kXLoadRows * kRowChunks / 32;
                constexpr int kRowsAtOnce = 32 / kRowChunks;
                const int lw = warp - kXLoadWarp;
                uint8_t *own = codes + (lw * 32 + lane) * 16;
                static_assert(kXLoadRows == kTile, "a place for a warp's rows");
                const uint8_t *keys = a.keys + static_cast<int64_t>(h) * D + 16 * (lane % kRowChunks);
                const int stride = a.Hkv * D, my_row = lane / kRowChunks;
                auto issue = [&](int i) {  // tile i (a commit group)
                    if (i < tiles) {
                        const int u = it + i, place = places[i * (kXRows / kTile) + lw];
                        const int left = place >= 0 ? L - (tok0 + i * kXRows + lw * kXLoadRows) : 0;  // rows that are there
                        const uint8_t *from = keys + static_cast<int64_t>(max(place, 0) + my_row) * stride;
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            cp_async_16_or_zero(own + ((u % kXCodes) * kPer + j) * (kXMmaWarp - kXLoadWarp) * 512,
                                                from + static_cast<int64_t>(j * kRowsAtOnce) * stride, j * kRowsAtOnce + my_row < left);
                    }
                    cp_async_commit();
                };
#pragma unroll
                for (int i = 0; i < kXAhead; ++i) issue(i);
                for (int i = 0; i < tiles && good; ++i) {
                    issue(i + kXAhead);
                    cp_async_wait<kXAhead>();
                    const int u = it + i, s = u % kXStages;
                    if (u >= kXStages) good = __all_sync(0xffffffffu, wait(&kempty[s], (u / kXStages - 1) & 1));
                    if (!good) break;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const int r = lw * kXLoadRows + j * kRowsAtOnce + lane / kRowChunks, c = lane % kRowChunks;
                        uint4 w[Chunk<F8>::kVecs];
                        const uint8_t *at = own + ((u % kXCodes) * kPer + j) * (kXMmaWarp - kXLoadWarp) * 512;
                        widen<F8>(*reinterpret_cast<const uint4 *>(at), w);
#pragma unroll
                        for (int v = 0; v < Chunk<F8>::kVecs; ++v) {
                            const int ch = c * Chunk<F8>::kVecs + v;
                            uint8_t *to = smem + s * X::kStageBytes + (ch >> 3) * (kXRows * kSubBytes) + swz128(r, ch & 7);
                            *reinterpret_cast<uint4 *>(to) = w[v];
                        }
                    }
                    mbar_arrive(&kfull[s]);
                }
                cp_async_wait<0>();
            }
        } else if (warp == kXMmaWarp) {
            if (lane == 0) {
                // (descriptors count 16 bytes: what is added to them is worked out before the loop)
                const uint64_t k0 = tc5::sw128_desc(smem, 16, 1024), q0 = tc5::sw128_desc(qs, 16, 1024);
                const uint32_t q_half = static_cast<uint32_t>(N * kSubBytes) >> 4;
                const uint32_t idesc = tc5::idesc_bf16_f32(kXRows, N, false, false, F8);
                for (int i = 0; i < tiles && good; ++i) {
                    const int u = it + i, s = u % kXStages, at = u & 1, turn = u >> 1;
                    // (tile u's sums go where those of tile u - 4 were)
                    good = wait(&kfull[s], (u / kXStages) & 1) && (turn == 0 || wait(&sfree[at], (turn - 1) & 1)) &&
                           (u < 4 || wait(&hfree[u & 3], ((u >> 2) - 1) & 1));
                    if (!good) break;
                    if (F8) fence_proxy_async_smem();  // (the generic proxy has written the keys)
                    tc5::fence_after_sync();
                    const uint64_t kd = k0 + static_cast<uint32_t>(s * (X::kStageBytes >> 4));
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        tc5::mma_bf16(tmem + at * width, kd + ((j >> 2) * (kXRows * kSubBytes) + (j & 3) * 32) / 16,
                                      q0 + (j >> 2) * q_half + (j & 3) * 2, idesc, j > 0);
                    tc5::commit(&sdone[at]);
                    tc5::commit(&kempty[s]);
                }
                if (!good) {  // let what was issued finish before TMEM is freed
                    tc5::commit(drain);
                    mbar_wait_bounded(drain, 0);
                }
            }
            __syncwarp();
        } else if (warp == kXFinalWarp) {
            // joins the groups' sums: four rows of a tile a lane, their old weights kXLook tiles ahead (one tile
            // ahead, every tile waits for memory's latency: 1.1 us)
            const int64_t base = (static_cast<int64_t>(b) * a.Hkv + h) * a.room;
            const int shift = a.ends ? a.ends[b] - L : 0;  // a token's position less its place
            float was[kXLook][4];
            auto look = [&](int i, float(&w)[4]) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = tok0 + i * kXRows + 32 * j + lane;
                    w[j] = final && i < tiles && tok < first_new ? a.old[base + tok] : 0.f;
                }
            };
#pragma unroll
            for (int i = 0; i < kXLook; ++i) look(i, was[i]);
            for (int i0 = 0; i0 < tiles && good; i0 += kXLook) {
#pragma unroll
                for (int ahead = 0; ahead < kXLook; ++ahead) {
                    const int i = i0 + ahead, u = it + i;
                    if (i >= tiles) break;
                    good = __all_sync(0xffffffffu, wait(&hdone[u & 3], (u >> 2) & 1));
                    if (!good) break;
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float *part_s = other + (u & 3) * kGroups * kXRows + 32 * j + lane;
                        v[j] = part_s[0];
#pragma unroll
                        for (int e = 1; e < kGroups; ++e) v[j] += part_s[e * kXRows];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&hfree[u & 3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = 32 * j + lane, tok = tok0 + i * kXRows + row;
                        if (!first) v[j] += sums[i * kXRows + row];
                        if (!final) {
                            sums[i * kXRows + row] = v[j];
                        } else if (tok < L) {
                            if (places[(i * kXRows + row) / kTile] < 0) v[j] = 0.f;
                            const bool fresh = tok >= first_new;
                            a.out[base + tok] = fresh ? v[j] : fmaf(a.decay, was[ahead][j], v[j]);
                            if (fresh && a.positions) a.positions[base + tok] = tok + shift;
                        }
                    }
                    look(i + kXLook, was[ahead]);
                }
            }
        } else {
            const int group = warp >> 2, r = 32 * (warp & 3) + (lane >> 2) + 8 * (lane & 3);  // the row that it ends with
            const int n0 = group * part, n1 = min(part, here - n0);
            uint64_t nl_r[XWarps<F8>::kPart / 8];  // -lse of this thread's columns, two by two
#pragma unroll
            for (int i = 0; i < XWarps<F8>::kPart / 8; ++i) {
                const int n = 8 * i + 2 * (lane & 3);
                nl_r[i] = pack2(n < n1 ? nl[n0 + n] : 0.f, n + 1 < n1 ? nl[n0 + n + 1] : 0.f);
            }
            for (int i = 0; i < tiles && good; ++i) {
                const int u = it + i, at = u & 1;
                // (a tile with new tokens has queries that do not see all of it)
                const bool all = !odd && tok0 + (i + 1) * kXRows <= first_new;
                good = __all_sync(0xffffffffu, wait(&sdone[at], (u >> 1) & 1));
                if (!good) break;
                tc5::fence_after_sync();
                const uint32_t rows = tc5::taddr(tmem, 32 * (warp & 3), at * width + n0);
                const int tok = tok0 + i * kXRows + 32 * (warp & 3);
                other[((u & 3) * kGroups + group) * kXRows + r] =
                    all ? row_sums<false, XWarps<F8>::kPart>(rows, n1, a.scale_log2, nl_r, last_s + n0, tok)
                        : row_sums<true, XWarps<F8>::kPart>(rows, n1, a.scale_log2, nl_r, last_s + n0, tok);
                tc5::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfree[at]), mbar_arrive(&hdone[u & 3]);
            }
        }
    }
    tc5::fence_before_sync();
    __syncthreads();
    if (warp == kXMmaWarp) tc5::tmem_free(tmem, tmem_cols);
}

template <bool F8, int D>
cudaError_t launch_weights(const WeightsArgs &a, int B, int64_t most, cudaStream_t stream) {
    const int64_t columns = static_cast<int64_t>(a.q_len) * a.G;
    if (columns <= kWFew) {
        // The pairs of a warp that take the least time by a model in microseconds: a CTA's start 4, each
        // pair at an SM's share of the memory (two CTAs an SM, 22 bytes a nanosecond each); rows three
        // quarters full, and, in waves, one more for the ends.  (8 x 4 rows of 4096 bf16 tokens: 1 pair 10.2
        // us, 2 8.3, 4 9.5; of 16384 1 29, 4 25, 8 24; 32 x 8 ragged FP8 rows 1 112, 4 68, 8 61; 16 pairs
        // were worse or the same.)  The lengths are not known here: rows much shorter than their tables get
        // more pairs than they need (8 x 4 rows of 4096 tokens in tables for 8192 9.5 us, 32768 9.8, 131072 14.9).
        const int64_t sms = sm_count();
        if (sms <= 0) return cudaErrorInvalidDevice;
        int pairs = 1;
        double least = 0.0;
        for (int n = 1; n <= 8; n *= 2) {
            const int64_t span = static_cast<int64_t>(n) * kWWarps * 2 * kTile;
            const double full = static_cast<double>((most + span - 1) / span) * a.Hkv * B / (2.0 * sms);
            const double cost = (full > 1.0 ? 0.75 * full + 1.0 : 1.0) * (4.0 + static_cast<double>(span) * D * (F8 ? 1 : 2) / 22e3);
            if (n == 1 || cost < least) least = cost, pairs = n;
        }
        const int64_t span = static_cast<int64_t>(pairs) * kWWarps * 2 * kTile;
        return launch_maybe_cooperative(columns <= 8 ? weights_kernel<F8, D, true> : weights_kernel<F8, D, false>,
                                        dim3(static_cast<unsigned>((most + span - 1) / span), a.Hkv, B), kWThreads, 0, stream,
                                        false, pdl_on(), a, pairs);
    }
    // 256 columns at a time, or shares of them that differ by little
    const int64_t chunks = (columns + kXColumns - 1) / kXColumns;
    const int n_most = static_cast<int>(((columns + chunks - 1) / chunks + 15) / 16 * 16);
    uint32_t cols = 64;  // of TMEM: two buffers, read 32 columns at a time
    while (cols < 2u * ((n_most + 31) / 32 * 32)) cols *= 2;
    // the tiles of a CTA: the fewest rounds of tiles over all SMs, a CTA's start counted as two
    const int64_t tiles = (most + kXRows - 1) / kXRows, rows = static_cast<int64_t>(a.Hkv) * B, sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int n = 1; n <= kXMostTiles; ++n) {
        const int64_t c = ((tiles + n - 1) / n * rows + sms - 1) / sms * (std::min<int64_t>(n, tiles) * chunks + 2);
        if (c < cost) cost = c, best = n;
    }
    auto kern = weights_tc_kernel<F8, D>;
    static std::atomic<uint64_t> smem_attr_done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(smem_attr_done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, XShape<F8, D>::bytes(kXColumns));
        if (e != cudaSuccess) return e;
        smem_attr_done.fetch_or(bit, std::memory_order_release);
    }
    CUtensorMap map{};
    if (!F8 && make_head_map(&map, a.keys, pa_cache_desc{a.num_blocks, a.block_size, a.Hkv, D}) != PA_OK)
        return cudaErrorUnknown;
    return launch_maybe_cooperative(kern, dim3(static_cast<unsigned>((tiles + best - 1) / best), a.Hkv, B), XWarps<F8>::kThreads,
                                    XShape<F8, D>::bytes(n_most), stream, false, pdl_on(), map, a, best, n_most, cols);
}

int weights_add(float *new_weights, const float *weights, int32_t *positions, const void *q, int32_t q_len, const float *lse,
                const void *k_cache, bool f8, const pa_cache_desc &cache, float scale, const int32_t *tables,
                int32_t max_blocks, const int32_t *lens, const int32_t *ends, int64_t room, int32_t B, int32_t Hq, float decay,
                int32_t *status, cudaStream_t stream) {
    if (B < 0 || q_len < 1 || q_len > 65535 || max_blocks <= 0 || room <= 0) return PA_EINVAL;
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (Hq <= 0 || Hq % cache.num_kv_heads != 0) return PA_EINVAL;
    if (!std::isfinite(scale) || !(decay >= 0.f) || !std::isfinite(decay)) return PA_EINVAL;
    if (Hq / cache.num_kv_heads > 32 || cache.num_kv_heads > 65535 || B > 65535) return PA_EUNSUPPORTED;
    if (static_cast<int64_t>(max_blocks) * cache.block_size > INT32_MAX / 2) return PA_EUNSUPPORTED;
    if (B == 0) return PA_OK;
    if (!new_weights || !weights || !q || !lse || !k_cache || !tables || !lens) return PA_EINVAL;
    if (!is_aligned(new_weights, 4) || !is_aligned(weights, 4) || !is_aligned(positions, 4) || !is_aligned(q, 16) ||
        !is_aligned(lse, 4) || !is_aligned(k_cache, 16) || !is_aligned(tables, 4) || !is_aligned(lens, 4) ||
        !is_aligned(ends, 4) || !is_aligned(status, 4))
        return PA_EINVAL;
    WeightsArgs a{};
    a.out = new_weights, a.old = weights, a.positions = positions, a.q = static_cast<const uint16_t *>(q), a.lse = lse;
    a.keys = static_cast<const uint8_t *>(k_cache), a.tables = tables, a.lens = lens, a.ends = ends, a.status = status;
    a.room = room, a.num_blocks = cache.num_blocks, a.block_size = cache.block_size, a.Hkv = cache.num_kv_heads;
    a.G = Hq / cache.num_kv_heads, a.q_len = q_len, a.max_blocks = max_blocks;
    a.scale_log2 = scale * 1.4426950408889634f, a.decay = decay;
    const int64_t most = std::min(static_cast<int64_t>(max_blocks) * cache.block_size, room);
    cudaError_t e;
    if (f8)
        e = cache.head_dim == 128 ? launch_weights<true, 128>(a, B, most, stream) : launch_weights<true, 64>(a, B, most, stream);
    else
        e = cache.head_dim == 128 ? launch_weights<false, 128>(a, B, most, stream) : launch_weights<false, 64>(a, B, most, stream);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_weights_add(float *new_weights, const float *weights, int32_t *positions, const void *q, int32_t q_len,
                   const float *lse, const void *k_cache, pa_cache_desc cache, const int32_t *block_tables,
                   int32_t max_blocks_per_seq, const int32_t *seq_lens, const int32_t *ends, int64_t room, int32_t B,
                   int32_t Hq, float scale, float decay, int32_t *status, pa_stream_t stream) {
    return pa::weights_add(new_weights, weights, positions, q, q_len, lse, k_cache, false, cache, scale, block_tables,
                           max_blocks_per_seq, seq_lens, ends, room, B, Hq, decay, status, stream);
}

int pa_weights_add_fp8(float *new_weights, const float *weights, int32_t *positions, const void *q, int32_t q_len,
                       const float *lse, const void *k_cache, pa_cache_desc cache, float k_scale,
                       const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                       const int32_t *ends, int64_t room, int32_t B, int32_t Hq, float scale, float decay,
                       int32_t *status, pa_stream_t stream) {
    if (!(k_scale > 0.f) || !std::isfinite(k_scale)) return PA_EINVAL;
    return pa::weights_add(new_weights, weights, positions, q, q_len, lse, k_cache, true, cache, scale * k_scale,
                           block_tables, max_blocks_per_seq, seq_lens, ends, room, B, Hq, decay, status, stream);
}

}  // extern "C"
