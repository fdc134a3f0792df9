// Eviction by accumulated attention weight (pa_cache_evict): of every layer, sequence
// and KV head, n tokens stay in the cache, the first n places of the sequence, and the
// blocks behind them are given back.
//
// The tokens that stay and stand below n are left where they are; the places below n that
// came free take the ones that stand behind, the k-th place the k-th token.  So a row
// is read only behind n and written only below it: nothing that moves meets anything
// else, in any order, and a call that is repeated does the same again.  No packing moves
// fewer rows.
//
// Two launches.  evict_lens_kernel works out every sequence's n, and writes the new
// lengths, tables and counts.  evict_kernel has a thread-block cluster per (layer,
// sequence, head): it finds the n-th largest weight over its shared memory (pa_topk.cuh),
// lists the free places and the tokens for them, and moves the rows.  Bound by the chain of the
// search where few tokens are thrown out (the 8 x 4 rows of a step, 64 of 1088 tokens each: 9.9 us);
// where many are (8 layers of 4 FP8 prompts of up to 16384 tokens: 68 us, half of the copy's rate for
// what is read and written) by the search, 24 us for all rows side by side, and then by memory.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_topk.cuh"

namespace pa {
namespace {

constexpr int kEvictMaxPools = 256;
constexpr int kLensThreads = 256;
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictCtas = 8;             // portable cluster size
constexpr int kEvictMaxSlice = 24576;     // tokens of a CTA
constexpr size_t kEvictSmemOfTwo = 113 * 1024;  // shared memory of a CTA of which two fit an SM
constexpr int kMoveTurns = 4;             // of a warp's ring of rows
constexpr uint32_t kSafe = 0xffffffffu;   // key of a token that stays whatever its weight

struct EvictArgs {
    int32_t *new_tables, *new_lens, *new_refs;
    const int32_t *tables, *lens, *refs;
    float *new_weights;            // [layers, B, Hkv, room]
    int32_t *new_positions;
    const float *weights;
    const int32_t *positions;
    int32_t *status;
    int64_t room;
    int32_t B, Hkv, max_blocks, num_blocks, block_size;
    int32_t budget, first, recent;
    int32_t ctas, slice, moves;    // of a cluster; tokens and moved rows of a CTA at most
    int32_t row_chunks;            // 16-byte chunks of one head's row in a pool
    uint8_t *pools[kEvictMaxPools];  // a layer's K and V in turn
};

// Entry j of a row's table that its L tokens use: a block in use, or -1.
__device__ __forceinline__ int used_entry(const EvictArgs &a, const int32_t *row, int j) {
    const int id = row[j];
    return id >= 0 && id < a.num_blocks && a.refs[id] > 0 ? id : -1;
}

// CTA b < B: sequence b's new length and table; the other CTAs copy the counts, a range each.
__global__ void __launch_bounds__(kLensThreads) evict_lens_kernel(const __grid_constant__ EvictArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x, bs = a.block_size;
    if (b >= a.B) {
        const int i = (b - a.B) * kLensThreads + tid;
        if (i < a.num_blocks) a.new_refs[i] = a.refs[i];
        return;
    }
    __shared__ int past_s, bad_s;   // entries up to the last block that others hold too; a bad entry or length
    const int most = a.max_blocks * bs;
    int L = a.lens[b];
    const bool bad_len = L < 0 || L > most || L > a.room;
    L = min(max(L, 0), most);
    if (tid == 0) past_s = 0, bad_s = bad_len;
    __syncthreads();
    const int32_t *row = a.tables + static_cast<int64_t>(b) * a.max_blocks;
    int32_t *out = a.new_tables + static_cast<int64_t>(b) * a.max_blocks;
    const int n_used = (L + bs - 1) / bs;
    int past = 0;
    bool bad = false;
    for (int j = tid; j < n_used; j += kLensThreads) {
        const int id = used_entry(a, row, j);
        if (id < 0) bad = true;
        else if (a.refs[id] > 1) past = j + 1;
    }
    if (past) atomicMax(&past_s, past);
    if (bad) bad_s = 1;
    __syncthreads();
    bad = bad_s;
    if (tid == 0 && bad) set_status(a.status, bad_len ? PA_STATUS_BAD_SEQLEN : PA_STATUS_BAD_BLOCK);
    const int fixed = min(L, past_s * bs);
    int64_t n = a.budget;
    if (fixed) n = max(n, static_cast<int64_t>(fixed) + a.first + a.recent);
    n = bad ? L : min(n, static_cast<int64_t>(L));
    if (tid == 0) a.new_lens[b] = static_cast<int>(n);
    // the block that a fork gave for the next token is the row's own, too
    const int next = L % bs == 0 && L < most ? used_entry(a, row, L / bs) : -1;
    const int stay = n < L ? static_cast<int>(n) / bs + 1 : n_used + (next >= 0);
    for (int j = tid; j < a.max_blocks; j += kLensThreads)
        out[j] = j < min(stay, n_used) ? used_entry(a, row, j) : j < stay ? next : -1;
}

// Words of shared memory for keys, and for the rows on their way.
__host__ __device__ constexpr int evict_keys(int slice) {
    return slice > kEvictWarps * kMoveTurns * 256 ? slice : kEvictWarps * kMoveTurns * 256;
}

// Rows src[p] -> dst[p], p < n (places of this head in both pools of a layer; in shared memory), by the
// CTA; kChunks: 16-byte chunks of a row.  A warp has kMoveTurns - 1 turns of 32 chunks of each pool on
// their way to its part of `stage`, from which every lane takes what it copied itself.  (Through
// registers, two turns at a time: the prompts 87 us; with 2 or 5 turns on their way 69 and 77.)
template <int kChunks>
__device__ __forceinline__ void move_rows(uint4 *k_pool, uint4 *v_pool, int Hkv, int h, const int32_t *src, const int32_t *dst,
                                          int n, uint4 *stage) {
    constexpr int kRows = 32 / kChunks, kStep = kEvictWarps * kRows;  // pairs of a turn, of all warps' turns
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p0 = warp * kRows + lane / kChunks, chunk = lane % kChunks;
    stage += warp * (kMoveTurns * 64) + lane;
    auto at = [&](int place) { return (static_cast<int64_t>(place) * Hkv + h) * kChunks + chunk; };
    auto issue = [&](int p, int slot) {
        if (p < n) {
            const int64_t x = at(src[p]);
            cp_async_16(stage + 64 * slot, k_pool + x);
            cp_async_16(stage + 64 * slot + 32, v_pool + x);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kMoveTurns - 1; ++i) issue(p0 + i * kStep, i);
    int slot = 0, next = kMoveTurns - 1;
    for (int p = p0; p < n; p += kStep) {
        issue(p + (kMoveTurns - 1) * kStep, next);
        cp_async_wait<kMoveTurns - 1>();
        const int64_t x = at(dst[p]);
        k_pool[x] = stage[64 * slot], v_pool[x] = stage[64 * slot + 32];
        slot = slot + 1 == kMoveTurns ? 0 : slot + 1, next = next + 1 == kMoveTurns ? 0 : next + 1;
    }
}

__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ __align__(16) uint8_t evict_smem[];
    TopkShared &sh = *reinterpret_cast<TopkShared *>(evict_smem);
    uint32_t *keys = reinterpret_cast<uint32_t *>(evict_smem + kTopkSharedBytes);
    int32_t *holes = reinterpret_cast<int32_t *>(keys + evict_keys(a.slice));   // this CTA's pairs: [moves] free places
    int32_t *movers = holes + a.moves;                              // ... and the tokens that take them
    __shared__ int past_s, newest_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bs = a.block_size;
    const int C = a.ctas, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t row = blockIdx.x / C;   // (layer, sequence, head)
    const int h = static_cast<int>(row % a.Hkv);
    const int b = static_cast<int>(row / a.Hkv % a.B), layer = static_cast<int>(row / a.Hkv / a.B);
    griddep_wait();
    griddep_launch_dependents();

    const int L = min(max(a.lens[b], 0), a.max_blocks * bs), n = a.new_lens[b];
    const int32_t *table = a.tables + static_cast<int64_t>(b) * a.max_blocks;
    const float *weights = a.weights + row * a.room;
    const int32_t *positions = a.positions + row * a.room;
    float *new_weights = a.new_weights + row * a.room;
    int32_t *new_positions = a.new_positions + row * a.room;
    const int thread = rank * kEvictThreads + tid, threads = C * kEvictThreads;
    if (n >= L) {  // nothing to throw out (or a row with a bad length or block, which is left as it is)
        const int all = static_cast<int>(min(static_cast<int64_t>(L), a.room));
        for (int t = thread; t < all; t += threads) new_weights[t] = weights[t], new_positions[t] = positions[t];
        return;
    }
    const int n_used = (L + bs - 1) / bs;
    if (layer == 0 && h == 0) {  // one cluster per sequence gives its blocks back
        for (int j = n / bs + 1 + thread; j < n_used; j += threads) atomicSub(&a.new_refs[table[j]], 1);
        if (thread == 0 && L % bs == 0 && L < a.max_blocks * bs) {
            const int next = used_entry(a, table, L / bs);
            if (next >= 0) atomicSub(&a.new_refs[next], 1);
        }
    }
    // tokens of blocks that others hold too, and those before them, stay in their places
    if (tid == 0) past_s = 0, newest_s = INT32_MIN;
    __syncthreads();
    int past = 0;
    for (int j = tid; j < n_used; j += kEvictThreads)
        if (a.refs[table[j]] > 1) past = j + 1;
    if (past) atomicMax(&past_s, past);
    const int per = ((L + C - 1) / C + 31) / 32 * 32;
    const int t0 = min(rank * per, L), mine = min(t0 + per, L) - t0;
    __syncthreads();
    const int fixed = past_s * bs;
    // Keys; and every place below n gets what it has now (a place that comes free gets another's, later).
    // The newest token stands in the last place, unless the row was cut and had no token since, which
    // the largest position tells: then the keys are made again (a pass for that position first would
    // read every row's positions twice; a step's rows 9.9 us, made again 10.5, the prompts' 68 and 73).
    Window seen;
    constexpr int kBatch = 4;  // loads on their way together (the stores would hold the next ones up)
    for (int newest = positions[L - 1];;) {
        seen = Window();
        int largest = INT32_MIN;
        for (int i0 = tid; i0 < mine; i0 += kBatch * kEvictThreads) {
            float w[kBatch];
            int p[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * kEvictThreads;
                w[j] = i < mine ? weights[t0 + i] : 0.f, p[j] = i < mine ? positions[t0 + i] : INT32_MIN;
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * kEvictThreads, t = t0 + i;
                if (i >= mine) break;
                largest = max(largest, p[j]);
                const bool safe = t < fixed || p[j] < a.first || p[j] > static_cast<int64_t>(newest) - a.recent;
                const uint32_t k = safe ? kSafe : float_key(w[j] == w[j] ? w[j] : INFINITY);
                keys[i] = k;
                seen.see(k, 0u, kSafe - 1u);
                if (t < n) new_weights[t] = w[j], new_positions[t] = p[j];
            }
        }
        __syncwarp();
        largest = __reduce_max_sync(0xffffffffu, largest);
        if (lane == 0) atomicMax(&newest_s, largest);
        meet(C);
        if (C > 1 && lane < C) largest = static_cast<int>(ld_shared_cluster_u32(map_shared_rank(smem_u32(&newest_s), lane)));
        largest = C > 1 ? __reduce_max_sync(0xffffffffu, largest) : newest_s;
        if (largest == newest) break;
        newest = largest;
    }

    auto key_at = [&](int i) { return keys[i]; };
    Border edge = cluster_threshold<kEvictThreads>(key_at, mine, seen, n, 0u, kSafe - 1u, C, sh, kTopkFew);
    edge = cluster_finish<kEvictThreads>(key_at, mine, edge, C, sh);
    const uint32_t border = edge.lo, need = edge.m == edge.inside ? ~0u : edge.m;

    // ---- which tokens stay: those above the border (or all from it on: none then counts as at it, or every one
    // does), and the first `need` at it.  Every warp's share is contiguous.
    const int share = ((mine + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
    const int i0 = min(warp * share, mine), i1 = min(i0 + share, mine);
    uint32_t counts[4] = {0, 0, 0, 0}, before[4], total[4];  // above, at the border; the same below n
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t above = keys[i] > border, at = keys[i] == border, low = t0 + i < n;
        counts[0] += above, counts[1] += at, counts[2] += above & low, counts[3] += at & low;
    }
    cluster_counts<kEvictThreads>(counts, C, sh, 0, before, total);
    const uint32_t kept_low = total[2] + min(total[3], need);  // of the first n
    const int pairs = n - static_cast<int>(kept_low);          // places that came free
    const int log_ctas = 31 - __clz(C);                        // pair p is CTA p % C's
    for (int i = i0; i < i1; i += 32) {
        const int t = t0 + i + lane;
        const bool here = i + lane < i1;
        const uint32_t k = here ? keys[i + lane] : 0u;
        const bool above = here && k > border, at = here && k == border;
        const uint32_t aboves = __ballot_sync(0xffffffffu, above), ats = __ballot_sync(0xffffffffu, at);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t tied = before[1] + __popc(ats & below);
        const uint32_t kept = before[0] + __popc(aboves & below) + min(tied, need);  // tokens that stay before this one
        const bool stays = above || (at && tied < need);
        if (here && stays != (t < n)) {
            const int p = static_cast<int>(t < n ? t - kept : kept - kept_low);
            int32_t *where = (t < n ? holes : movers) + (p >> log_ctas);
            if (C > 1) st_shared_cluster_u32(map_shared_rank(smem_u32(where), p & (C - 1)), static_cast<uint32_t>(t));
            else *where = t;
        }
        before[0] += __popc(aboves), before[1] += __popc(ats);
    }
    meet(C);

    // ---- the rows
    const int my_pairs = (pairs - rank + C - 1) >> log_ctas;
    // their places, and the weights and positions of the tokens that move
    for (int p0 = tid; p0 < my_pairs; p0 += kBatch * kEvictThreads) {
        float w[kBatch];
        int pos[kBatch], to[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int p = p0 + j * kEvictThreads;
            if (p >= my_pairs) break;
            const int from = movers[p];
            to[j] = holes[p];
            w[j] = weights[from], pos[j] = positions[from];
            movers[p] = table[from / bs] * bs + from % bs;
            holes[p] = table[to[j] / bs] * bs + to[j] % bs;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (p0 + j * kEvictThreads < my_pairs) new_weights[to[j]] = w[j], new_positions[to[j]] = pos[j];
    }
    __syncthreads();
    uint4 *k_pool = reinterpret_cast<uint4 *>(a.pools[2 * layer]), *v_pool = reinterpret_cast<uint4 *>(a.pools[2 * layer + 1]);
    uint4 *stage = reinterpret_cast<uint4 *>(keys);  // (the keys have been used)
    if (a.row_chunks == 16) move_rows<16>(k_pool, v_pool, a.Hkv, h, movers, holes, my_pairs, stage);
    else if (a.row_chunks == 8) move_rows<8>(k_pool, v_pool, a.Hkv, h, movers, holes, my_pairs, stage);
    else move_rows<4>(k_pool, v_pool, a.Hkv, h, movers, holes, my_pairs, stage);
}

size_t evict_smem_bytes(int slice, int moves) {
    return kTopkSharedBytes + static_cast<size_t>(evict_keys(slice)) * 4 + static_cast<size_t>(moves) * 8;
}
// Rows that a sequence of up to `most` tokens moves, per CTA of C: no more than there are tokens behind the
// new length n, or below it that may leave (n less those that others hold, at most the budget).
int evict_moves(int64_t most, int budget, int C) {
    return static_cast<int>((std::min<int64_t>(budget, most / 2) + C - 1) / C + 1) / 2 * 2;
}
int evict_slice(int64_t most, int C) { return static_cast<int>(((most + C - 1) / C + 31) / 32 * 32); }

}  // namespace
}  // namespace pa

extern "C" int pa_cache_evict(int32_t *new_tables, int32_t *new_lens, int32_t *new_refs, float *new_weights,
                              int32_t *new_positions, const int32_t *tables, const int32_t *lens, const int32_t *refs,
                              const float *weights, const int32_t *positions, int64_t room, int32_t B,
                              int32_t max_blocks_per_seq, void *const *pools, int32_t n_pools, int32_t elem_bytes,
                              pa_cache_desc cache, int32_t budget, int32_t first, int32_t recent, int32_t *status,
                              pa_stream_t stream) {
    if (B < 0 || max_blocks_per_seq <= 0 || room <= 0 || budget < 1 || first < 0 || recent < 0) return PA_EINVAL;
    if (static_cast<int64_t>(first) + recent > budget) return PA_EINVAL;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_EINVAL;
    const int rc = pa::check_cache(cache);
    if (rc) return rc;
    if (!pools || n_pools < 2 || n_pools % 2) return PA_EINVAL;
    if (n_pools > pa::kEvictMaxPools) return PA_EUNSUPPORTED;
    for (int i = 0; i < n_pools; ++i)
        if (!pools[i] || !pa::is_aligned(pools[i], 16)) return PA_EINVAL;
    if (static_cast<int64_t>(max_blocks_per_seq) * cache.block_size > INT32_MAX / 2) return PA_EUNSUPPORTED;
    if (!new_refs || !refs || new_refs == refs) return PA_EINVAL;
    if (B > 0 && (!new_tables || !new_lens || !new_weights || !new_positions || !tables || !lens || !weights || !positions))
        return PA_EINVAL;
    if (B > 0 && (new_tables == tables || new_lens == lens || new_weights == weights || new_positions == positions))
        return PA_EINVAL;
    for (const void *p : {static_cast<const void *>(new_tables), static_cast<const void *>(new_lens),
                          static_cast<const void *>(new_refs), static_cast<const void *>(new_weights),
                          static_cast<const void *>(new_positions), static_cast<const void *>(tables),
                          static_cast<const void *>(lens), static_cast<const void *>(refs),
                          static_cast<const void *>(weights), static_cast<const void *>(positions),
                          static_cast<const void *>(status)})
        if (!pa::is_aligned(p, 4)) return PA_EINVAL;
    const int64_t most = std::min(room, static_cast<int64_t>(max_blocks_per_seq) * cache.block_size);
    const int64_t rows = static_cast<int64_t>(n_pools / 2) * B * cache.num_kv_heads;
    if (most > static_cast<int64_t>(pa::kEvictCtas) * pa::kEvictMaxSlice || B > 65535 ||
        rows > INT32_MAX / pa::kEvictCtas)
        return PA_EUNSUPPORTED;
    pa::EvictArgs a{};
    a.new_tables = new_tables, a.new_lens = new_lens, a.new_refs = new_refs;
    a.tables = tables, a.lens = lens, a.refs = refs;
    a.new_weights = new_weights, a.new_positions = new_positions, a.weights = weights, a.positions = positions;
    a.status = status, a.room = room, a.B = B, a.Hkv = cache.num_kv_heads, a.max_blocks = max_blocks_per_seq;
    a.num_blocks = cache.num_blocks, a.block_size = cache.block_size;
    a.budget = budget, a.first = first, a.recent = recent;
    a.row_chunks = cache.head_dim * elem_bytes / 16;
    for (int i = 0; i < n_pools; ++i) a.pools[i] = static_cast<uint8_t *>(pools[i]);
    // One CTA per row where it can be: its meetings and passes cost half of a cluster's, and more rows are
    // under way at once (256 rows of 16384 tokens: 1 CTA 67 us, 2 76, 4 92).  More where two would not fit
    // an SM, and, of long rows, where there are few.  (By the room, the lengths are not known here: a
    // step's 32 rows of 1088 tokens 9.9 us, with room for 4096 12.5, for 16384 and more 19.)
    const int sms = pa::sm_count();
    if (sms <= 0) return PA_ECUDA;
    a.ctas = 1;
    while (a.ctas < pa::kEvictCtas &&
           (pa::evict_smem_bytes(pa::evict_slice(most, a.ctas), pa::evict_moves(most, budget, a.ctas)) > pa::kEvictSmemOfTwo ||
            (most >= 4096 * a.ctas && 2 * rows * a.ctas <= 2 * sms)))
        a.ctas *= 2;
    a.slice = pa::evict_slice(most, a.ctas), a.moves = pa::evict_moves(most, budget, a.ctas);
    const int copies = (cache.num_blocks + pa::kLensThreads - 1) / pa::kLensThreads;
    if (pa::launch_maybe_cooperative(pa::evict_lens_kernel, dim3(B + copies), pa::kLensThreads, 0, stream, false, pa::pdl_on(),
                                     a) != cudaSuccess)
        return PA_ECUDA;
    if (B == 0) return PA_OK;
    static std::atomic<uint64_t> smem_attr_done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(smem_attr_done.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(pa::evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(pa::evict_smem_bytes(pa::kEvictMaxSlice, pa::kEvictMaxSlice / 2 + 2))) != cudaSuccess)
            return PA_ECUDA;
        smem_attr_done.fetch_or(bit, std::memory_order_release);
    }
    const cudaError_t e = pa::launch_clustered(pa::evict_kernel, dim3(static_cast<unsigned>(rows * a.ctas)), a.ctas,
                                               pa::kEvictThreads, static_cast<int>(pa::evict_smem_bytes(a.slice, a.moves)), stream,
                                               pa::pdl_on(), a);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}
