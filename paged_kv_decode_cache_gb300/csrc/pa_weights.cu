// The attention weight that cached tokens draw (pa_weights_add): for every sequence,
// KV head and token t
//   w[t] <- decay w[t] + sum over the queries i and the group's heads g that see t of
//           exp(scale <q_ig, K_t> - lse_ig),
// the softmax's own probabilities, rebuilt from the log-sum-exp that attention gave.  Every
// key is read once; a token's sum belongs to one warp, so no atomics and the same bits
// every time.
#include <algorithm>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"

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
constexpr int kWTiles = 2;                              // wide kernel: tiles of 16 tokens of a warp
constexpr int kWTokens = kWWarps * kWTiles * kTile;     // ... tokens of a CTA
constexpr int kWColumns = 128;                          // ... columns in shared memory at once

// Columns c0 .. c0 + here - 1 of a (sequence, KV head) into shared memory: the MMA's operands,
// the lse in log2 units, and the last token that each sees (-1: none).
template <bool F8, int D>
__device__ __forceinline__ void load_columns(const WeightsArgs &a, int b, int h, int first_new, int c0, int here, uint4 *qs,
                                             float *lse_s, int *last_s) {
    constexpr int kVecs = D / 32;
    const int tiles = (here + 7) / 8;
    for (int i = threadIdx.x; i < tiles * kVecs * 32; i += kWThreads) {
        const int ln = i & 31, v = (i >> 5) % kVecs, col = (i >> 5) / kVecs * 8 + (ln >> 2);
        const int64_t row = (static_cast<int64_t>(b) * a.q_len + (c0 + col) / a.G) * a.Hkv * a.G + h * a.G + (c0 + col) % a.G;
        uint4 w = col < here ? *reinterpret_cast<const uint4 *>(a.q + row * D + vec_dim<F8>(v, ln & 3))
                             : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (F8)
            w = make_uint4(to_f16x2(bf16lo(w.x), bf16hi(w.x)), to_f16x2(bf16lo(w.y), bf16hi(w.y)),
                           to_f16x2(bf16lo(w.z), bf16hi(w.z)), to_f16x2(bf16lo(w.w), bf16hi(w.w)));
        qs[i] = w;
    }
    for (int col = threadIdx.x; col < tiles * 8; col += kWThreads) {
        const int i = (c0 + col) / a.G;
        const int64_t row = (static_cast<int64_t>(b) * a.q_len + i) * a.Hkv * a.G + h * a.G + (c0 + col) % a.G;
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
// that old and new weights are whole lines.
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
    const int stride = a.Hkv * kRowBytes;                  // between rows (check_cache: below 2^31)
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
    load_columns<F8, D>(a, b, h, first_new, 0, columns, qs, lse_s, last_s);
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

// More columns: a CTA per 256 tokens of a (sequence, KV head), 32 to a warp, whose keys it keeps
// in registers while the columns (query, head of the group) pass through shared memory, up
// to 128 at a time.
template <bool F8, int D>
__global__ void __launch_bounds__(kWThreads, 2) weights_wide_kernel(const WeightsArgs a) {
    constexpr int kRowBytes = D * (F8 ? 1 : 2);
    constexpr int kChunks = kRowBytes / 64;
    constexpr int kVecs = kChunks * Chunk<F8>::kVecs;
    extern __shared__ uint4 qs[];                       // [column tiles][kVecs][32 lanes]
    __shared__ float lse_s[kWColumns];                  // in log2 units
    __shared__ int last_s[kWColumns];                   // last token that the column sees, -1: none
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
    const int tok0 = static_cast<int>(blockIdx.x) * kWTokens;
    if (tok0 >= L) return;
    const int n_cols = a.q_len * a.G, first_new = L - a.q_len;

    // ---- this warp's keys
    uint4 raw[kWTiles][2][kChunks];
    const int w0 = tok0 + warp * kWTiles * kTile;
    bool there[kWTiles];
#pragma unroll
    for (int i = 0; i < kWTiles; ++i) {
        const int at = w0 + i * kTile;
        there[i] = at < L;
        int phys = 0;
        if (there[i]) {
            phys = a.tables[static_cast<int64_t>(b) * a.max_blocks + at / bs];
            if (phys < 0 || phys >= a.num_blocks) {
                if (lane == 0 && h == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
                there[i] = false;
                phys = 0;
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int tok = at + g + 8 * r;
            const bool ok = there[i] && tok < L;
            const uint8_t *row = a.keys + ((static_cast<int64_t>(phys) * bs + tok % bs) * a.Hkv + h) * kRowBytes + 16 * t;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) raw[i][r][c] = ok ? load_once(row + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
    }

    // ---- the columns
    float sum[kWTiles][2] = {};
    for (int c0 = 0; c0 < n_cols; c0 += kWColumns) {
        const int here = min(kWColumns, n_cols - c0), tiles = (here + 7) / 8;
        if (c0) __syncthreads();
        load_columns<F8, D>(a, b, h, first_new, c0, here, qs, lse_s, last_s);
        __syncthreads();
        for (int nt = 0; nt < tiles; ++nt) {
            float acc[kWTiles][4] = {};
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                uint4 w[Chunk<F8>::kVecs];
#pragma unroll
                for (int k = 0; k < Chunk<F8>::kVecs; ++k) w[k] = qs[(nt * kVecs + c * Chunk<F8>::kVecs + k) * 32 + lane];
#pragma unroll
                for (int i = 0; i < kWTiles; ++i) {
                    uint4 x[Chunk<F8>::kVecs], y[Chunk<F8>::kVecs];
                    widen<F8>(raw[i][0][c], x);
                    widen<F8>(raw[i][1][c], y);
#pragma unroll
                    for (int k = 0; k < Chunk<F8>::kVecs; ++k) {
                        mma_16x8x16<F8>(acc[i], x[k].x, y[k].x, x[k].y, y[k].y, w[k].x, w[k].y);
                        mma_16x8x16<F8>(acc[i], x[k].z, y[k].z, x[k].w, y[k].w, w[k].z, w[k].w);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kWTiles; ++i)
                add_columns(sum[i], acc[i], a.scale_log2, lse_s + nt * 8 + 2 * t, last_s + nt * 8 + 2 * t, w0 + i * kTile + g);
        }
    }

    // ---- the four lanes of a token, and what it had
    const int64_t base = (static_cast<int64_t>(b) * a.Hkv + h) * a.room;
    const int shift = a.ends ? a.ends[b] - L : 0;  // a token's position less its place
#pragma unroll
    for (int i = 0; i < kWTiles; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float s = sum[i][r];
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            const int tok = w0 + i * kTile + g + 8 * r;
            if (t != 0 || tok >= L) continue;
            if (!there[i]) s = 0.f;
            const bool fresh = tok >= first_new;
            a.out[base + tok] = fresh ? s : fmaf(a.decay, a.old[base + tok], s);
            if (fresh && a.positions) a.positions[base + tok] = tok + shift;
        }
}

template <bool F8, int D>
cudaError_t launch_weights(const WeightsArgs &a, int B, int64_t most, cudaStream_t stream) {
    const int64_t columns = static_cast<int64_t>(a.q_len) * a.G;
    if (columns <= kWFew) {
        // long runs of tokens, but CTAs for four waves and more
        const int64_t all = (most + 2 * kTile - 1) / (2 * kTile) * a.Hkv * B, sms = sm_count();
        int pairs = 1;
        while (pairs < 16 && all >= 2 * pairs * kWWarps * 8 * sms) pairs *= 2;
        const int64_t span = static_cast<int64_t>(pairs) * kWWarps * 2 * kTile;
        return launch_maybe_cooperative(columns <= 8 ? weights_kernel<F8, D, true> : weights_kernel<F8, D, false>,
                                        dim3(static_cast<unsigned>((most + span - 1) / span), a.Hkv, B), kWThreads, 0, stream,
                                        false, pdl_on(), a, pairs);
    }
    const int smem = static_cast<int>((std::min<int64_t>(kWColumns, columns) + 7) / 8 * 8) * D * 2;
    return launch_maybe_cooperative(weights_wide_kernel<F8, D>,
                                    dim3(static_cast<unsigned>((most + kWTokens - 1) / kWTokens), a.Hkv, B), kWThreads, smem,
                                    stream, false, pdl_on(), a);
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
