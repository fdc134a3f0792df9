// Pages of the cache: sequences forked, reordered and dropped with copy on
// write (pa_sequences_fork), live blocks moved to the front of the pools
// (pa_blocks_compact), blocks copied (pa_blocks_copy).
//
// The state is functional: new tables, lengths and reference counts are
// written whole beside the old ones, so a call can be captured and repeated.
// A planning kernel works out what goes where (integers only; the lowest free
// ids are given out in row order, so that the result does not depend on
// scheduling), and one copy kernel moves the pages of all pools.
//
// The planning kernel is ONE thread-block cluster: its phases need every
// earlier write, and a cluster barrier costs a fraction of a launch or a
// grid-wide wait.  Shared counters are L2 atomics on integers, whose order
// cannot show.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxPlanCtas = 8;        // portable cluster size
constexpr int kMaxRows = 4096;         // sequences per fork
constexpr int kMaxPools = 256;
constexpr int kCopyThreads = 256;
constexpr int kPiece = 16 * 1024;      // bytes of a block per CTA and turn
constexpr int kOwnTurns = 16;          // turns of a copy that a lone planning CTA makes itself
constexpr int kNearBlocks = 2048;     // blocks whose compaction is planned by every CTA
constexpr int kPlanWords = 2048;       // words of counts and tables per planning CTA
// A fork that one CTA plans in shared memory: rows, and words of counts and tables (64 rows,
// 6700 words: 10.0 us, with a cluster of 4 11.5; 112 rows, 4900 words: 12.4 and 11.7).
constexpr int kNearRows = 64, kNearWords = 8192;

// Block-wide exclusive prefix sum over kThreads threads; *total gets the sum.  (T: two
// counts in one 64-bit number share the shuffles and the barriers.)
template <int kThreads = kPlanThreads, typename T = int>
__device__ __forceinline__ T block_scan(T v, T *warp_sums, T *total) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T s = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < kWarps) warp_sums[lane] = s;
    }
    __syncthreads();
    const T before = warp ? warp_sums[warp - 1] : 0;
    *total = warp_sums[kWarps - 1];
    __syncthreads();  // (warp_sums is free again)
    return before + x - v;
}

// The CTAs' values of a cluster: *before gets the sum of those below this one, the result is the
// sum of all.  `mine` in shared memory, which the caller keeps until the next cluster barrier.
__device__ __forceinline__ int cluster_scan(int *mine, int value, int ctas, int *before) {
    if (threadIdx.x == 0) *mine = value;
    cluster_sync();
    const int lane = threadIdx.x & 31, rank = static_cast<int>(cluster_ctarank());
    int v = 0;
    if (lane < ctas) v = __float_as_int(ld_shared_cluster(map_shared_rank(smem_u32(mine), lane)));
    *before = __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
    return __reduce_add_sync(0xffffffffu, v);
}

// What a plan hands to the copy kernel.
struct CopyList {
    int32_t count;      // entries used
    int32_t pad[3];
    // int4 entries follow: source block, destination block, token rows
};

struct CopyArgs {
    const CopyList *list;       // the copies, or:
    const int2 *pairs;          // (source, destination), n of them, whole blocks
    int n_pairs;
    int n_pools;
    int row_bytes;              // of a token
    int block_size, num_blocks;
    int32_t *status;
    // tables to rewrite while at it (pa_blocks_compact), or null
    int32_t *new_tables;
    const int32_t *tables, *lens, *remap;
    int64_t *new_slots;         // and the next tokens' slots, or null
    const int64_t *slots;
    int B, max_blocks;
    uint8_t *pools[kMaxPools];
};

// Turns first, first + step, ... of a copy.  A turn is 16 KB of one block of one
// pool, copied by one CTA with four 16-byte loads per thread (of kCopyThreads) in
// flight.  entry(k): the k-th copy's source (< 0: none), destination and token rows.
template <int kThreads, typename Entry>
__device__ __forceinline__ void copy_turns(const CopyArgs &a, int count, int first, int step, Entry &&entry) {
    constexpr int kEach = kPiece / 16 / kThreads;
    const int64_t block_bytes = static_cast<int64_t>(a.block_size) * a.row_bytes;
    const int pieces = static_cast<int>((block_bytes + kPiece - 1) / kPiece);
    const int64_t turns = static_cast<int64_t>(count) * a.n_pools * pieces;
#pragma unroll 4
    for (int64_t t = first; t < turns; t += step) {
        const int piece = static_cast<int>(t % pieces);
        const int64_t u = t / pieces;
        const int pool = static_cast<int>(u % a.n_pools);
        const int4 e = entry(static_cast<int>(u / a.n_pools));
        const int src = e.x, dst = e.y, rows = e.z;
        if (src < 0) continue;
        const int64_t from = static_cast<int64_t>(piece) * kPiece;
        const int64_t left = static_cast<int64_t>(rows) * a.row_bytes - from;
        if (left <= 0) continue;
        const int vecs = static_cast<int>((left < kPiece ? left : static_cast<int64_t>(kPiece)) / 16);
        const uint4 *in = reinterpret_cast<const uint4 *>(a.pools[pool] + src * block_bytes + from);
        uint4 *out = reinterpret_cast<uint4 *>(a.pools[pool] + dst * block_bytes + from);
        uint4 v[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int x = i * kThreads + threadIdx.x;
            if (x < vecs) v[i] = __ldcs(in + x);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int x = i * kThreads + threadIdx.x;
            if (x < vecs) __stcs(out + x, v[i]);
        }
    }
}

// A plan's list as entries of a copy.
struct Listed {
    const CopyList *list;
    __device__ __forceinline__ int4 operator()(int k) const { return __ldcg(reinterpret_cast<const int4 *>(list + 1) + k); }
};

struct ForkArgs {
    int32_t *new_tables, *new_lens, *new_refs;
    int64_t *slots;
    const int32_t *tables, *lens, *refs, *parents;
    int32_t *status;
    CopyList *list;
    int32_t *free_list;   // [B_new] the lowest free ids
    int32_t *tail_count;  // [num_blocks] new rows whose next token goes into it
    int32_t *tail_first;  // [num_blocks] the first of them
    int B_old, B_new, max_blocks, num_blocks, block_size;
};

__device__ __forceinline__ int checked_len(int L, int lmax, int32_t *status) {
    if (L >= 0 && L <= lmax) return L;
    set_status(status, PA_STATUS_BAD_SEQLEN);
    return L < 0 ? 0 : lmax;
}

// The block that a row of length L (checked, below the table's tokens) has for its next
// token, `entry` being its table's entry L / bs: its partial last block, or the one that
// a fork gave it and that no token has gone into yet, which is in use; else -1.
__device__ __forceinline__ int next_block(int entry, int L, int bs, const int32_t *refs, int num_blocks) {
    if (entry < 0 || entry >= num_blocks) return -1;
    return L % bs || refs[entry] > 0 ? entry : -1;
}

// The number of free ids a thread's segment [lo, hi) of the counts holds.
__device__ __forceinline__ int count_zero(const int32_t *refs, int lo, int hi) {
    int n = 0;
    for (int i = lo; i < hi; ++i) n += __ldcg(refs + i) == 0;
    return n;
}

// f(entry, block id) for a table row's first n entries, by one warp, four loads
// per lane in flight.
template <typename F>
__device__ __forceinline__ void for_entries(const int32_t *row, int n, int lane, F &&f) {
    for (int e0 = lane; e0 < n; e0 += 128) {
        int id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) id[u] = e0 + 32 * u < n ? __ldg(row + e0 + 32 * u) : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (e0 + 32 * u < n) f(e0 + 32 * u, id[u]);
    }
}

// Row i of the new state is row parents[i] of the old one, sharing its blocks.
// An old row with c children changes every count of its blocks by c - 1, so
// rows with one child (most of them) touch no count.  Then the block of the
// next token, position L: its partial last block, or the empty one that an earlier
// fork gave it.  A row keeps it when every reference to it is some new row's block
// for the next token and this is the first such row; any other row takes a free block
// in its place and copies its rows, if any; so does a row that ends with a full block.
// kSmall: one CTA, which keeps the counts and lists in shared memory, so that only the
// first loads, the tables and the copies themselves wait for memory (4 beams of a
// request: 9.7 -> 6.0 us).  `copy.list`: the plan's, for a copy so small that this CTA makes
// it itself; null: another launch does.
template <bool kSmall>
__global__ void __launch_bounds__(kPlanThreads)
fork_plan_kernel(const ForkArgs a, const __grid_constant__ CopyArgs copy) {
    extern __shared__ int32_t smem[];
    int32_t *row_parent = smem;                     // [B_new], -1: no sequence
    int32_t *row_len = row_parent + a.B_new;        // [B_new]
    int32_t *row_tail = row_len + a.B_new;          // [B_new] the block for its next token (next_block)
    int32_t *row_rank = row_tail + a.B_new;         // [B_new] needs a block: which one; else -1
    int32_t *children = row_rank + a.B_new;         // [B_old]
    int32_t *old_len = children + a.B_old;          // [B_old]
    int32_t *near = old_len + a.B_old;              // kSmall: the arrays below
    int32_t *refs = kSmall ? near : a.new_refs;                            // [num_blocks]
    int32_t *tail_count = kSmall ? near + a.num_blocks : a.tail_count;      // [num_blocks]
    int32_t *tail_first = kSmall ? near + 2 * a.num_blocks : a.tail_first;  // [num_blocks]
    int32_t *free_list = kSmall ? near + 3 * a.num_blocks : a.free_list;    // [B_new]
    auto get = [](const int32_t *p) { return kSmall ? *p : __ldcg(p); };   // (what other CTAs write is read from L2)
    auto everyone = [] {
        if (kSmall) __syncthreads();
        else cluster_sync();
    };
    __shared__ uint64_t warp_sums[32];
    __shared__ int cta_free;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    const int cta = kSmall ? 0 : blockIdx.x, ctas = kSmall ? 1 : gridDim.x;
    const int gid = cta * kPlanThreads + tid, gthreads = ctas * kPlanThreads;
    const int bs = a.block_size, mb = a.max_blocks, lmax = mb * bs;

    // ---- the rows' parents and lengths (every CTA for itself), the counts copied
    // (each thread's first loads are asked for at once)
    const int len0 = tid < a.B_old ? a.lens[tid] : 0, parent0 = tid < a.B_new ? a.parents[tid] : -1;
    const int refs0 = gid < a.num_blocks ? a.refs[gid] : 0;
    for (int j = tid; j < a.B_old; j += kPlanThreads) {
        children[j] = 0;
        old_len[j] = checked_len(j == tid ? len0 : a.lens[j], lmax, a.status);
    }
    for (int i = tid; i < a.B_new; i += kPlanThreads) row_parent[i] = i == tid ? parent0 : a.parents[i];
    for (int i = gid; i < a.num_blocks; i += gthreads) {
        refs[i] = i == gid ? refs0 : a.refs[i];
        if (kSmall) tail_count[i] = 0, tail_first[i] = INT32_MAX;
    }
    __syncthreads();
    for (int i = tid; i < a.B_new; i += kPlanThreads) {
        int p = row_parent[i], L = 0, t = -1;
        if (p >= a.B_old) {
            set_status(a.status, PA_STATUS_BAD_PARENT);
            p = -1;
        }
        if (p >= 0) {
            L = old_len[p];
            atomicAdd(children + p, 1);
            if (L < lmax) t = next_block(a.tables[static_cast<int64_t>(p) * mb + L / bs], L, bs, a.refs, a.num_blocks);
            if (!kSmall && cta == 0 && t >= 0) tail_count[t] = 0, tail_first[t] = INT32_MAX;
        }
        row_parent[i] = p < 0 ? -1 : p;
        row_len[i] = L;
        row_tail[i] = t;
    }
    everyone();

    // ---- references dropped and added; tables copied (a warp per row)
    for (int j = gid >> 5; j < a.B_old; j += gthreads >> 5) {
        const int change = children[j] - 1, L = old_len[j];
        if (change == 0) continue;
        for_entries(a.tables + static_cast<int64_t>(j) * mb, min(L / bs + 1, mb), lane, [&](int e, int id) {
            if (e * bs >= L) id = next_block(id, L, bs, a.refs, a.num_blocks);   // (past a full block; -1 is no fault there)
            else if (id < 0 || id >= a.num_blocks) set_status(a.status, PA_STATUS_BAD_BLOCK);
            if (id >= 0 && id < a.num_blocks) atomicAdd(refs + id, change);
        });
    }
    for (int i = gid >> 5; i < a.B_new; i += gthreads >> 5) {
        const int p = row_parent[i], nb = (row_len[i] + bs - 1) / bs + (row_len[i] % bs == 0 && row_tail[i] >= 0);
        int32_t *row = a.new_tables + static_cast<int64_t>(i) * mb;
        if (lane == 0 && row_tail[i] >= 0) {
            atomicAdd(tail_count + row_tail[i], 1);
            atomicMin(tail_first + row_tail[i], i);
        }
        for_entries(a.tables + static_cast<int64_t>(max(p, 0)) * mb, nb, lane, [&](int e, int id) {
            if (id < 0 || id >= a.num_blocks) {
                set_status(a.status, PA_STATUS_BAD_BLOCK);
                id = -1;
            }
            row[e] = id;
        });
        for (int e = nb + lane; e < mb; e += 32) row[e] = -1;
    }
    everyone();

    // ---- which rows need a block (every CTA for itself, in row order), and the lowest
    // free ids: each CTA a slice, each thread a segment.  What both read is asked
    // for at once, and both are counted in one scan.
    const int per_row = (a.B_new + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(tid * per_row, a.B_new), i1 = min(i0 + per_row, a.B_new);
    const int slice = (a.num_blocks + ctas - 1) / ctas;
    const int s0 = min(cta * slice, a.num_blocks), s1 = min(s0 + slice, a.num_blocks);
    const int seg = (slice + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(s0 + tid * seg, s1), hi = min(lo + seg, s1);
    uint32_t mine = 0, mine_free = 0;   // rows that need a block, and << 16 those that copy into it; free ids
    uint64_t zero = 0;                  // the segment's first 64 ids: free or not
    for (int i = i0; i < i1; ++i) {
        const int L = row_len[i], t = row_tail[i];
        const int makers = t >= 0 ? get(tail_count + t) : 0, all = t >= 0 ? get(refs + t) : 0;
        const int first = t >= 0 ? get(tail_first + t) : 0;
        int need = row_parent[i] >= 0 && L % bs == 0 && L < lmax && t < 0;
        if (t >= 0 && !(makers == all && first == i)) need = L % bs ? 1 | 1 << 16 : 1;
        row_rank[i] = need;
        mine += need;
    }
    for (int j = lo; j < hi; j += 4) {
        int count[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) count[u] = j + u < hi ? get(refs + j + u) : 1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (count[u] == 0) {
                ++mine_free;
                if (j + u - lo < 64) zero |= 1ull << (j + u - lo);
            }
    }
    uint64_t total;
    const uint64_t before = block_scan<kPlanThreads, uint64_t>(static_cast<uint64_t>(mine_free) << 32 | mine, warp_sums, &total);
    const int needed = total & 0xffff, copies = static_cast<int>(total >> 16 & 0xffff);
    uint32_t rank_at = static_cast<uint32_t>(before);
    for (int i = i0; i < i1; ++i) {
        const int need = row_rank[i];
        row_rank[i] = need ? static_cast<int>(rank_at) : -1;  // its block's rank, and << 16 its copy's
        rank_at += need;
    }
    int n_free = static_cast<int>(total >> 32);
    if (needed > 0) {  // (the same in every CTA)
        int at = static_cast<int>(before >> 32);
        if (!kSmall) {
            int below;
            n_free = cluster_scan(&cta_free, n_free, ctas, &below);
            at += below;
        }
        for (; zero && at < needed; zero &= zero - 1) free_list[at++] = lo + __ffsll(static_cast<long long>(zero)) - 1;
        for (int j = lo + 64; j < hi && at < needed; ++j)
            if (get(refs + j) == 0) free_list[at++] = j;
        everyone();
    } else {
        __syncthreads();
    }

    // ---- the rows' last blocks, slots and copies
    int4 *entries = reinterpret_cast<int4 *>(a.list + 1);
    if (gid == 0) a.list->count = copies;
    for (int i = gid; i < a.B_new; i += gthreads) {
        const int L = row_len[i], off = L % bs, e = L / bs, tail = row_tail[i];
        int64_t slot = -1;
        if (row_rank[i] >= 0) {
            const int rank = row_rank[i] & 0xffff;
            int id = -1;
            if (rank < n_free) {
                id = get(free_list + rank);
                a.new_tables[static_cast<int64_t>(i) * mb + e] = id;
                refs[id] = 1;
                if (tail >= 0) atomicSub(refs + tail, 1);
                slot = static_cast<int64_t>(id) * bs + off;
            } else {
                set_status(a.status, PA_STATUS_NO_BLOCKS);
            }
            if (off) entries[row_rank[i] >> 16] = make_int4(id < 0 ? -1 : tail, id, off, 0);
        } else if (row_parent[i] >= 0) {
            if (tail >= 0) slot = static_cast<int64_t>(tail) * bs + off;
            else if (L == lmax) set_status(a.status, PA_STATUS_BAD_SEQLEN);  // the table is full
        }
        a.slots[i] = slot;
        a.new_lens[i] = L;
    }
    if (kSmall) {
        __syncthreads();
        for (int i = tid; i < a.num_blocks; i += kPlanThreads) a.new_refs[i] = refs[i];
        if (copy.list) copy_turns<kPlanThreads>(copy, copies, 0, 1, Listed{copy.list});
    }
}

struct CompactArgs {
    int32_t *new_tables, *new_refs, *remap, *n_live;
    const int32_t *tables, *lens, *refs;
    int32_t *status;
    CopyList *list;
    int32_t *holes;       // [num_blocks] free ids below the live count, ascending
    int B, max_blocks, num_blocks, block_size;
};

// With n live blocks of which A already lie below n, the n - A others move to
// the n - A free ids below n, both in ascending order.  A block's rank among
// the live ones gives both lists' indices: live id >= n has rank r - A, free id
// below n has rank id - r.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
    __shared__ int32_t warp_sums[32];
    __shared__ int cta_live;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x;
    const int slice = (a.num_blocks + ctas - 1) / ctas;
    const int s0 = min(cta * slice, a.num_blocks), s1 = min(s0 + slice, a.num_blocks);
    const int seg = (slice + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(s0 + tid * seg, s1), hi = min(lo + seg, s1);
    int total, below;
    int rank = block_scan(hi - lo - count_zero(a.refs, lo, hi), warp_sums, &total);
    const int n = cluster_scan(&cta_live, total, ctas, &below);
    rank += below;
    // ---- what stays, the holes, and how many blocks move
    int r = rank;
    for (int i = lo; i < hi; ++i) {
        const int refs = a.refs[i];
        if (i == n) a.list->count = n - r;
        if (refs != 0) {
            if (i < n) {
                a.remap[i] = i;
                a.new_refs[i] = refs;
            }
            ++r;
        } else {
            a.remap[i] = -1;
            if (i < n) a.holes[i - r] = i;
        }
        if (i >= n) a.new_refs[i] = 0;
    }
    if (cta == 0 && tid == 0) {
        *a.n_live = n;
        if (n == a.num_blocks) a.list->count = 0;
    }
    cluster_sync();
    // ---- the moves
    int4 *entries = reinterpret_cast<int4 *>(a.list + 1);
    const int first = n - __ldcg(&a.list->count);  // A
    r = rank;
    for (int i = lo; i < hi; ++i) {
        const int refs = a.refs[i];
        if (refs == 0) continue;
        if (i >= n) {
            const int to = __ldcg(a.holes + (r - first));
            entries[r - first] = make_int4(i, to, a.block_size, 0);
            a.remap[i] = to;
            a.new_refs[to] = refs;
        }
        ++r;
    }
}

// Rewrites the tables, and the slots if there are any; new_id(id): where a block of the
// pool went, or -1.  A row's entries are those of its tokens and, where its length is a
// multiple of the block size, the block in use that a fork gave it for its next token.
template <typename NewId>
__device__ __forceinline__ void rewrite_tables(const CopyArgs &a, NewId &&new_id) {
    const int64_t n = static_cast<int64_t>(a.B) * a.max_blocks;
    for (int64_t x = blockIdx.x * static_cast<int64_t>(kCopyThreads) + threadIdx.x; x < n;
         x += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int b = static_cast<int>(x / a.max_blocks), e = static_cast<int>(x % a.max_blocks);
        const int L = checked_len(a.lens[b], a.max_blocks * a.block_size, a.status);
        int id = -1;
        if (e * a.block_size <= L) {
            id = a.tables[x];
            id = id >= 0 && id < a.num_blocks ? new_id(id) : -1;
            if (id < 0 && e * a.block_size < L) set_status(a.status, PA_STATUS_BAD_BLOCK);
        }
        a.new_tables[x] = id;
    }
    if (!a.slots) return;
    for (int b = blockIdx.x * kCopyThreads + threadIdx.x; b < a.B; b += gridDim.x * kCopyThreads) {
        const int64_t slot = a.slots[b], block = slot / a.block_size;
        int id = -1;
        if (slot >= 0) {
            if (block < a.num_blocks) id = new_id(static_cast<int>(block));
            if (id < 0) set_status(a.status, PA_STATUS_BAD_SLOT);
        }
        a.new_slots[b] = id < 0 ? -1 : static_cast<int64_t>(id) * a.block_size + slot % a.block_size;
    }
}

// Moves the listed blocks' first rows in every pool.  CTAs take turns in a
// stride, so that the list's length (which only the GPU knows) spreads over all of
// them.  Destinations are free blocks and sources live ones, so turns never meet.
template <bool kPairs>
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    if (kPairs) {
        copy_turns<kCopyThreads>(a, a.n_pairs, blockIdx.x, gridDim.x, [&](int k) {
            const int2 e = a.pairs[k];
            const bool bad = e.x >= 0 && (e.x >= a.num_blocks || e.y < 0 || e.y >= a.num_blocks);
            if (bad && threadIdx.x == 0) set_status(a.status, PA_STATUS_BAD_BLOCK);
            return make_int4(bad ? -1 : e.x, e.y, a.block_size, 0);
        });
    } else {
        if (a.new_tables) rewrite_tables(a, [&](int id) { return a.remap[id]; });
        copy_turns<kCopyThreads>(a, a.list->count, blockIdx.x, gridDim.x, Listed{a.list});
    }
}

// The plan and the copy in one launch, for pools of up to kNearBlocks blocks: every CTA
// makes the plan for itself in shared memory (2 us, the counts being a few KB in
// L2; a second launch and the way through memory are 2.5) and takes its turns
// of the copy; the first one writes the new counts.
__global__ void __launch_bounds__(kCopyThreads)
compact_near_kernel(const CompactArgs a, const __grid_constant__ CopyArgs copy) {
    constexpr int kEach = kNearBlocks / kCopyThreads;   // ids per thread
    __shared__ int32_t warp_sums[kCopyThreads / 32];
    __shared__ int32_t remap[kNearBlocks], holes[kNearBlocks / 2], movers[kNearBlocks / 2];
    __shared__ int32_t stay;   // live blocks that keep their id
    griddep_wait();
    griddep_launch_dependents();
    const int first_id = threadIdx.x * kEach, nb = a.num_blocks;
    int refs[kEach], live = 0, n;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        refs[u] = first_id + u < nb ? a.refs[first_id + u] : 0;
        live += refs[u] != 0;
    }
    const int rank = block_scan<kCopyThreads>(live, warp_sums, &n);
    if (threadIdx.x == 0 && n == nb) stay = n;
    int r = rank;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int i = first_id + u;
        if (i >= nb) break;
        if (i == n) stay = r;
        if (refs[u] == 0) {
            remap[i] = -1;
            if (i < n) holes[i - r] = i;   // (at most n and nb - n of them)
        } else {
            if (i < n) remap[i] = i;
            ++r;
        }
    }
    __syncthreads();
    const int moves = n - stay;
    r = rank;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int i = first_id + u;
        if (i < nb && refs[u] != 0) {
            if (i >= n) {
                const int k = r - stay;
                movers[k] = i;
                remap[i] = holes[k];
            }
            ++r;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *a.n_live = n;
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int i = first_id + u;
            if (i >= nb) break;
            a.remap[i] = remap[i];
            if (i >= n) a.new_refs[i] = 0;
            if (refs[u] != 0) a.new_refs[remap[i]] = refs[u];
        }
    }
    if (copy.new_tables) rewrite_tables(copy, [&](int id) { return remap[id]; });
    copy_turns<kCopyThreads>(copy, moves, blockIdx.x, gridDim.x,
                             [&](int k) { return make_int4(movers[k], holes[k], a.block_size, 0); });
}

int check_pools(void *const *pools, int32_t n_pools, int32_t elem_bytes, const pa_cache_desc &c) {
    if (n_pools < 0 || (n_pools > 0 && !pools)) return PA_EINVAL;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_EINVAL;
    const int rc = check_cache(c);
    if (rc) return rc;
    if (n_pools > kMaxPools) return PA_EUNSUPPORTED;
    if (static_cast<int64_t>(c.num_kv_heads) * c.head_dim * elem_bytes > (1 << 24)) return PA_EUNSUPPORTED;
    for (int i = 0; i < n_pools; ++i)
        if (!pools[i] || !is_aligned(pools[i], 16)) return PA_EINVAL;
    return PA_OK;
}

void set_pools(CopyArgs &a, void *const *pools, int32_t n_pools, int32_t elem_bytes, const pa_cache_desc &c,
               int32_t *status) {
    a.n_pools = n_pools;
    a.row_bytes = c.num_kv_heads * c.head_dim * elem_bytes;
    a.block_size = c.block_size;
    a.num_blocks = c.num_blocks;
    a.status = status;
    for (int i = 0; i < n_pools; ++i) a.pools[i] = static_cast<uint8_t *>(pools[i]);
}

// Enough CTAs for `turns` (an upper bound), at most eight resident per SM.
template <typename... Args>
int launch_turns(void (*kernel)(Args...), int64_t turns, cudaStream_t stream, const Args &...args) {
    const int sms = sm_count();
    if (sms <= 0) return PA_ECUDA;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(turns, static_cast<int64_t>(sms) * 8));
    const cudaError_t e = launch_maybe_cooperative(kernel, dim3(static_cast<unsigned>(grid)), kCopyThreads, 0, stream,
                                                   false, pdl_on(), args...);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

int64_t pieces_of(const pa_cache_desc &c, int32_t elem_bytes) {
    const int64_t bytes = static_cast<int64_t>(c.block_size) * c.num_kv_heads * c.head_dim * elem_bytes;
    return (bytes + kPiece - 1) / kPiece;
}

// CTAs of a planning cluster: one per kPlanWords words it reads, up to eight.
int plan_ctas(int64_t words) {
    int n = 1;
    while (n < kMaxPlanCtas && words > kPlanWords * static_cast<int64_t>(n)) n *= 2;
    return n;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_fork_workspace_bytes(int32_t B_old, int32_t B_new, int32_t num_blocks) {
    if (B_old < 0 || B_new < 0 || num_blocks <= 0) return 0;
    return pa::up(sizeof(pa::CopyList) + 16 * static_cast<size_t>(B_new)) + pa::up(4 * static_cast<size_t>(B_new)) +
           2 * pa::up(4 * static_cast<size_t>(num_blocks));
}

size_t pa_compact_workspace_bytes(int32_t num_blocks) {
    if (num_blocks <= 0) return 0;
    return pa::up(sizeof(pa::CopyList) + 16 * static_cast<size_t>(num_blocks)) +
           pa::up(4 * static_cast<size_t>(num_blocks));
}

int pa_sequences_fork(int32_t *new_tables, int32_t *new_lens, int32_t *new_refs, int64_t *slot_mapping,
                      const int32_t *tables, const int32_t *lens, const int32_t *refs, const int32_t *parents,
                      int32_t B_old, int32_t B_new, int32_t max_blocks_per_seq, void *const *pools, int32_t n_pools,
                      int32_t elem_bytes, pa_cache_desc cache, void *workspace, size_t workspace_bytes,
                      int32_t *status, pa_stream_t stream) {
    if (B_old < 0 || B_new < 0 || max_blocks_per_seq <= 0) return PA_EINVAL;
    int rc = pa::check_pools(pools, n_pools, elem_bytes, cache);
    if (rc) return rc;
    if (B_old > pa::kMaxRows || B_new > pa::kMaxRows) return PA_EUNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * cache.block_size > INT32_MAX / 2) return PA_EUNSUPPORTED;
    if (!new_refs || !refs || (B_old > 0 && (!tables || !lens)) ||
        (B_new > 0 && (!new_tables || !new_lens || !slot_mapping || !parents)))
        return PA_EINVAL;
    if (new_refs == refs || (B_new > 0 && (new_tables == tables || new_lens == lens))) return PA_EINVAL;
    for (const void *p : {static_cast<const void *>(new_tables), static_cast<const void *>(new_lens),
                          static_cast<const void *>(new_refs), static_cast<const void *>(tables),
                          static_cast<const void *>(lens), static_cast<const void *>(refs),
                          static_cast<const void *>(parents)})
        if (!pa::is_aligned(p, 4)) return PA_EINVAL;
    if (!pa::is_aligned(slot_mapping, 8)) return PA_EINVAL;
    if (!workspace || workspace_bytes < pa_fork_workspace_bytes(B_old, B_new, cache.num_blocks) ||
        !pa::is_aligned(workspace, 256))
        return PA_EWORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    auto take = [&](size_t bytes) {
        uint8_t *p = ws;
        ws += pa::up(bytes);
        return p;
    };
    pa::ForkArgs a{};
    a.new_tables = new_tables, a.new_lens = new_lens, a.new_refs = new_refs, a.slots = slot_mapping;
    a.tables = tables, a.lens = lens, a.refs = refs, a.parents = parents, a.status = status;
    a.list = reinterpret_cast<pa::CopyList *>(take(sizeof(pa::CopyList) + 16 * static_cast<size_t>(B_new)));
    a.free_list = reinterpret_cast<int32_t *>(take(4 * static_cast<size_t>(B_new)));
    a.tail_count = reinterpret_cast<int32_t *>(take(4 * static_cast<size_t>(cache.num_blocks)));
    a.tail_first = reinterpret_cast<int32_t *>(take(4 * static_cast<size_t>(cache.num_blocks)));
    a.B_old = B_old, a.B_new = B_new, a.max_blocks = max_blocks_per_seq;
    a.num_blocks = cache.num_blocks, a.block_size = cache.block_size;
    const int64_t words = cache.num_blocks + static_cast<int64_t>(B_old + B_new) * max_blocks_per_seq;
    const bool small = words <= pa::kNearWords && std::max(B_old, B_new) <= pa::kNearRows;
    const int ctas = small ? 1 : std::max(2, pa::plan_ctas(words));
    const int64_t turns = static_cast<int64_t>(B_new) * n_pools * pa::pieces_of(cache, elem_bytes);
    const bool own_copy = small && turns <= pa::kOwnTurns;
    pa::CopyArgs c{};
    pa::set_pools(c, pools, n_pools, elem_bytes, cache, status);
    c.list = own_copy ? a.list : nullptr;
    int smem = (4 * B_new + 2 * B_old) * 4;
    if (small) smem += (3 * cache.num_blocks + B_new) * 4;
    auto kern = small ? pa::fork_plan_kernel<true> : pa::fork_plan_kernel<false>;
    static std::atomic<uint64_t> smem_attr_done[2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(smem_attr_done[small].load(std::memory_order_acquire) & bit)) {
        const int most = small ? 7 * pa::kNearRows + 3 * pa::kNearWords : 6 * pa::kMaxRows;   // words
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most * 4) != cudaSuccess)
            return PA_ECUDA;
        smem_attr_done[small].fetch_or(bit, std::memory_order_release);
    }
    if (pa::launch_clustered(kern, dim3(ctas), ctas, pa::kPlanThreads, smem, stream, pa::pdl_on(), a, c) != cudaSuccess)
        return PA_ECUDA;
    if (turns == 0 || own_copy) return PA_OK;
    c.list = a.list;
    return pa::launch_turns(pa::copy_blocks_kernel<false>, turns, stream, c);
}

int pa_blocks_compact(int32_t *new_tables, int32_t *new_refs, int32_t *remap, int32_t *n_live, const int32_t *tables,
                      const int32_t *lens, const int32_t *refs, int32_t B, int32_t max_blocks_per_seq,
                      void *const *pools, int32_t n_pools, int32_t elem_bytes, pa_cache_desc cache, void *workspace,
                      size_t workspace_bytes, int32_t *status, pa_stream_t stream) {
    return pa_blocks_compact_slots(new_tables, new_refs, remap, n_live, nullptr, tables, lens, refs, nullptr, B,
                                   max_blocks_per_seq, pools, n_pools, elem_bytes, cache, workspace, workspace_bytes,
                                   status, stream);
}

int pa_blocks_compact_slots(int32_t *new_tables, int32_t *new_refs, int32_t *remap, int32_t *n_live,
                            int64_t *new_slots, const int32_t *tables, const int32_t *lens, const int32_t *refs,
                            const int64_t *slots, int32_t B, int32_t max_blocks_per_seq, void *const *pools,
                            int32_t n_pools, int32_t elem_bytes, pa_cache_desc cache, void *workspace,
                            size_t workspace_bytes, int32_t *status, pa_stream_t stream) {
    if (B < 0 || max_blocks_per_seq <= 0) return PA_EINVAL;
    int rc = pa::check_pools(pools, n_pools, elem_bytes, cache);
    if (rc) return rc;
    if (static_cast<int64_t>(max_blocks_per_seq) * cache.block_size > INT32_MAX / 2) return PA_EUNSUPPORTED;
    if (!new_refs || !remap || !n_live || !refs || (B > 0 && (!new_tables || !tables || !lens))) return PA_EINVAL;
    if (new_refs == refs || remap == refs || remap == new_refs) return PA_EINVAL;
    if (!new_slots != !slots || (slots && new_slots == slots)) return PA_EINVAL;
    if (!pa::is_aligned(slots, 8) || !pa::is_aligned(new_slots, 8)) return PA_EINVAL;
    for (const void *p : {static_cast<const void *>(new_tables), static_cast<const void *>(new_refs),
                          static_cast<const void *>(remap), static_cast<const void *>(n_live),
                          static_cast<const void *>(tables), static_cast<const void *>(lens),
                          static_cast<const void *>(refs)})
        if (!pa::is_aligned(p, 4)) return PA_EINVAL;
    if (!workspace || workspace_bytes < pa_compact_workspace_bytes(cache.num_blocks) ||
        !pa::is_aligned(workspace, 256))
        return PA_EWORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    pa::CompactArgs a{};
    a.new_tables = new_tables, a.new_refs = new_refs, a.remap = remap, a.n_live = n_live;
    a.tables = tables, a.lens = lens, a.refs = refs, a.status = status;
    a.list = reinterpret_cast<pa::CopyList *>(ws);
    ws += pa::up(sizeof(pa::CopyList) + 16 * static_cast<size_t>(cache.num_blocks));
    a.holes = reinterpret_cast<int32_t *>(ws);
    a.B = B, a.max_blocks = max_blocks_per_seq, a.num_blocks = cache.num_blocks, a.block_size = cache.block_size;
    pa::CopyArgs c{};
    pa::set_pools(c, pools, n_pools, elem_bytes, cache, status);
    c.list = a.list;
    if (B > 0) c.new_tables = new_tables, c.new_slots = new_slots, c.slots = slots;
    c.tables = tables, c.lens = lens, c.remap = remap, c.B = B, c.max_blocks = max_blocks_per_seq;
    // (at most half of the blocks move)
    const int64_t turns = std::max(static_cast<int64_t>(cache.num_blocks / 2) * n_pools * pa::pieces_of(cache, elem_bytes),
                                   static_cast<int64_t>(B) * max_blocks_per_seq / pa::kCopyThreads);
    if (cache.num_blocks <= pa::kNearBlocks) return pa::launch_turns(pa::compact_near_kernel, turns, stream, a, c);
    const int ctas = pa::plan_ctas(cache.num_blocks);
    if (pa::launch_clustered(pa::compact_plan_kernel, dim3(ctas), ctas, pa::kPlanThreads, 0, stream, pa::pdl_on(), a) !=
        cudaSuccess)
        return PA_ECUDA;
    if (B == 0 && n_pools == 0) return PA_OK;
    return pa::launch_turns(pa::copy_blocks_kernel<false>, turns, stream, c);
}

int pa_blocks_copy(void *const *pools, int32_t n_pools, int32_t elem_bytes, pa_cache_desc cache, const int32_t *pairs,
                   int32_t n_pairs, int32_t *status, pa_stream_t stream) {
    if (n_pairs < 0) return PA_EINVAL;
    int rc = pa::check_pools(pools, n_pools, elem_bytes, cache);
    if (rc) return rc;
    if (n_pairs == 0 || n_pools == 0) return PA_OK;
    if (!pairs || !pa::is_aligned(pairs, 8)) return PA_EINVAL;
    pa::CopyArgs c{};
    pa::set_pools(c, pools, n_pools, elem_bytes, cache, status);
    c.pairs = reinterpret_cast<const int2 *>(pairs);
    c.n_pairs = n_pairs;
    const int64_t turns = static_cast<int64_t>(n_pairs) * n_pools * pa::pieces_of(cache, elem_bytes);
    return pa::launch_turns(pa::copy_blocks_kernel<true>, turns, stream, c);
}

}  // extern "C"
