// Beam search's selection: the K best continuations of every request over its
// beams and the vocabulary, in one launch that reads the logits once.
//
//   score(w, v) = cum_w + (x_wv - lse_w),  lse_w = max + ln sum_v exp(x_wv - max)
//
// Within a row the scores are ordered as the logits, so one pass over a
// row's logits gives both its (max, sum) and its K largest logits; lse enters
// only when the rows of a request are joined.  A CTA takes a slice of a row, in chunks
// that it holds in registers: 4 16-byte vectors per thread, all in flight at once.
// The K-th largest of the first chunk's thread maxima bounds the K-th largest
// value from below, so that only about K of a chunk's 8192 values ever leave the
// registers, into a pool in shared memory; no warp waits for another until the
// pool is a quarter full, when its K best raise the bound.  The last CTA of a
// request to finish joins its lists.
//
// Sums: exp in fp32 from x - max (exact for bf16), fp32 sums of 8 per vector
// and of a thread's vectors, 64 bits across threads and slices.  Scores are
// compared in 64 bits: bf16 logits repeat, and beams' scores come close to one
// another, so a score rounded to fp32 could trade two candidates.
#include <cuda_bf16.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                      // 16-byte vectors per thread and chunk
constexpr int kChunkVecs = kThreads * kVecs;
constexpr int kMaxK = 64;
constexpr int kMaxBeams = 64;
constexpr int kMaxJoin = 4096;                // candidates a request's join holds
constexpr int kPool = 2 * kThreads;            // candidates of a slice at a time
constexpr int kTargetCtas = 8 * 152;          // slices: about 8 CTAs per SM
constexpr int kMinSliceVecs = 2 * kThreads;   // and no smaller than two vectors per thread

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
    // NaN -> -inf, two bf16 values or one fp32
    __device__ static uint32_t clean(uint32_t w) {
        if constexpr (k16) {
            const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&w),
                                             __nv_bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80)));
            return *reinterpret_cast<const uint32_t *>(&x);
        } else {
            return __float_as_uint(fmaxf(__uint_as_float(w), -INFINITY));
        }
    }
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
    __device__ static float max(const uint4 &v) {
        if constexpr (k16) {
            auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
            const __nv_bfloat162 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            return fmaxf(fmaxf(get(v, 0), get(v, 1)), fmaxf(get(v, 2), get(v, 3)));
        }
    }
};

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

struct Candidate {
    float x;
    int32_t v;  // vocabulary entry, -1: none
};
__device__ __forceinline__ bool before(const Candidate &a, const Candidate &b) {
    return a.x > b.x || (a.x == b.x && a.v < b.v);
}

struct BeamArgs {
    float *scores;
    int32_t *tokens, *parents;
    const void *logits;
    int64_t row_stride;
    const float *cum;
    const uint8_t *finished;
    int32_t eos;
    int beams, vocab, K, slices;
    int32_t *tickets;      // [groups], zero between calls
    float *part_max;       // [rows, slices]
    double *part_sum;      // [rows, slices]
    Candidate *part_list;  // [rows, slices, K]
};

// A row's vectors: vector i holds entries i E .. i E + E - 1, whatever the row's
// alignment, so that equal rows give equal sums to the last bit.  A row that starts
// `skew` bytes past a 16-byte boundary takes each vector from two aligned ones.
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
    template <int W>
    __device__ void load_skewed(uint4 (&raw)[kVecs], int i0, int end) const {  // skew = 4 W + (0 or 2) bytes
        const int bits = (skew & 3) * 8;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = i0 + j * kThreads;
            if (i >= end || i >= whole) continue;
            const uint4 lo = __ldg(grid + i), hi = __ldg(grid + i + 1);
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            raw[j] = make_uint4(__funnelshift_r(w[W], w[W + 1], bits), __funnelshift_r(w[W + 1], w[W + 2], bits),
                                __funnelshift_r(w[W + 2], w[W + 3], bits), __funnelshift_r(w[W + 3], w[W + 4], bits));
        }
    }
    // Vectors i0, i0 + kThreads, ... below end, NaN as -inf, and -inf past the end.
    __device__ void load(uint4 (&raw)[kVecs], int i0, int end) const {
        using V = Vec<T>;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) raw[j] = make_uint4(V::kFill, V::kFill, V::kFill, V::kFill);
        if (skew == 0) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int i = i0 + j * kThreads;
                if (i < end && i < whole) raw[j] = __ldcs(grid + i);
            }
        } else if (skew < 4) {
            load_skewed<0>(raw, i0, end);
        } else if (skew < 8) {
            load_skewed<1>(raw, i0, end);
        } else if (skew < 12) {
            load_skewed<2>(raw, i0, end);
        } else {
            load_skewed<3>(raw, i0, end);
        }
        if (i0 + (kVecs - 1) * kThreads >= whole) {  // the row's end: entry by entry
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int i = i0 + j * kThreads;
                if (i < whole || i >= end) continue;
                uint32_t w[4] = {V::kFill, V::kFill, V::kFill, V::kFill};
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (i * E + e < vocab) V::put(w, e, x[i * E + e]);
                raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            raw[j] = make_uint4(V::clean(raw[j].x), V::clean(raw[j].y), V::clean(raw[j].z), V::clean(raw[j].w));
    }
};

// The largest key that at least K of the threads' keys reach (0: fewer than K
// do), bit by bit from the top; a CTA-wide count per bit.
template <int kKeyLow>
__device__ __forceinline__ uint32_t kth_key(uint32_t mine, int K) {
    uint32_t key = 0u;
    for (int bit = 31; bit >= kKeyLow; --bit)
        if (__syncthreads_count(mine >= (key | 1u << bit)) >= K) key |= 1u << bit;
    return key;
}

// pool[0 .. n) reduced to its min(n, K) first candidates, in order: an entry's
// place is the number of entries before it.  n <= 2 kThreads.
__device__ __forceinline__ int keep_first(Candidate *pool, int n, int K) {
    Candidate c[2];
    int place[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = u * kThreads + threadIdx.x;
        place[u] = K;
        if (i < n) {
            c[u] = pool[i];
            int before_it = 0;
            for (int j = 0; j < n; ++j) before_it += before(pool[j], c[u]);
            place[u] = before_it;
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
__device__ __noinline__ int exact_slice(const Row<T> &row, int v0, int v1, int K, Candidate *pool, int *count) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    const int tid = threadIdx.x;
    int kept = 0;
    float floor = -INFINITY;   // values at or below it are not among the K largest
    for (int c0 = v0; c0 < v1; c0 += kChunkVecs) {
        uint4 raw[kVecs];
        row.load(raw, c0 + tid, v1);
        auto each = [&](auto &&f) {  // f(value, vocabulary entry) of this thread's values above the floor
            for (int j = 0; j < kVecs; ++j)
                for (int e = 0; e < E; ++e) {
                    const float v = V::get(raw[j], e);
                    if (v > floor) f(v, (c0 + j * kThreads + tid) * E + e);
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
            if (at < kPool) pool[at] = Candidate{v, i};
        });
        __syncthreads();
        kept = keep_first(pool, min(*count, kPool), K);
        if (kept == K) floor = pool[K - 1].x;
    }
    return kept;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamArgs a) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    extern __shared__ uint64_t join_keys[];  // [beams * slices * K], then as many int32 (the join)
    __shared__ Candidate pool[kPool];        // candidates for the slice's K largest
    __shared__ int count, ticket;
    __shared__ float red_max[kThreads / 32];
    __shared__ double red_sum[kThreads / 32];
    __shared__ double lse[kMaxBeams];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row_id = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
    const int group = row_id / a.beams, K = a.K;
    const bool done = a.finished && a.finished[row_id];

    if (!done) {
        const Row<T> row(static_cast<const T *>(a.logits) + row_id * a.row_stride, a.vocab);
        const int vecs = (a.vocab + E - 1) / E;
        const int per = (vecs + a.slices - 1) / a.slices;
        const int v0 = min(slice * per, vecs), v1 = min(v0 + per, vecs);
        const int period = max(1, kPool / 3 / K);   // chunks between looks at the pool
        float m = -INFINITY, sum = 0.f;   // this thread's maximum and sum of exp(x - m)
        float cut = -INFINITY;            // values below it, or with `strict` at it, are not among the K largest
        bool strict = true, overfull = false;
        if (tid == 0) count = 0;
        __syncthreads();
        int chunk = 0;
        for (int c0 = v0; c0 < v1; c0 += kChunkVecs, ++chunk) {
            uint4 raw[kVecs];
            row.load(raw, c0 + tid, v1);
            float vmax[kVecs], cmax = -INFINITY;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                vmax[j] = V::max(raw[j]);
                cmax = fmaxf(cmax, vmax[j]);
            }
            // ---- sum of exponentials
            if (cmax > m) {
                sum *= fast_exp2((m - cmax) * 1.4426950408889634f);  // (m = -inf: 0)
                m = cmax;
            }
            if (m > -INFINITY) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    float s[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) s[e] = fast_exp2((V::get(raw[j], e) - m) * 1.4426950408889634f);
#pragma unroll
                    for (int o = E / 2; o > 0; o >>= 1)
#pragma unroll
                        for (int e = 0; e < o; ++e) s[e] += s[e + o];
                    sum += s[0];
                }
            }
            // ---- candidates: the first chunk's bound is the K-th largest of its threads' maxima
            if (chunk == 0) {
                const uint32_t key = kth_key<V::kKeyLow>(cmax > -INFINITY ? order_key(cmax) : 0u, K);
                if (key) {
                    cut = key_value<V::kKeyLow>(key);
                    strict = false;
                }
            }
            auto passes = [&](float v) { return strict ? v > cut : v >= cut; };
            if (passes(cmax)) {
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    if (!passes(vmax[j])) continue;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float v = V::get(raw[j], e);
                        if (!passes(v)) continue;
                        const int at = atomicAdd(&count, 1);
                        if (at < kPool) pool[at] = Candidate{v, (c0 + j * kThreads + tid) * E + e};
                    }
                }
            }
            if (chunk % period == period - 1) {  // raise the bound before the pool fills
                __syncthreads();
                const int n = count;
                __syncthreads();
                if (n > kPool) {
                    overfull = true;
                    cut = INFINITY, strict = true;
                } else if (n > kPool / 4) {
                    const int kept = keep_first(pool, n, K);
                    if (tid == 0) count = kept;
                    if (kept == K) {
                        cut = pool[K - 1].x;   // (later entries of an equal value come after it)
                        strict = true;
                    }
                    __syncthreads();
                }
            }
        }
        __syncthreads();
        int kept;
        if (overfull || count > kPool) kept = exact_slice<T>(row, v0, v1, K, pool, &count);
        else kept = keep_first(pool, count, K);
        // ---- the slice's maximum, sum and list
        float top = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) red_max[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, red_max[i]);
        double z = m > -INFINITY ? static_cast<double>(sum * fast_exp2((m - top) * 1.4426950408889634f)) : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) red_sum[warp] = z;
        __syncthreads();
        const int64_t part = static_cast<int64_t>(row_id) * a.slices + slice;
        if (tid == 0) {
            double s = 0.0;
            for (int i = 0; i < kThreads / 32; ++i) s += red_sum[i];
            a.part_max[part] = top;
            a.part_sum[part] = s;
        }
        if (tid < K) a.part_list[part * K + tid] = tid < kept ? pool[tid] : Candidate{-INFINITY, -1};
    }

    // ---- the request's last CTA joins its rows' slices
    __threadfence();
    __syncthreads();
    if (tid == 0) ticket = atomicAdd(a.tickets + group, 1);
    __syncthreads();
    if (ticket != a.beams * a.slices - 1) return;
    __threadfence();
    if (tid == 0) a.tickets[group] = 0;
    const int first_row = group * a.beams;
    if (tid < a.beams) {
        double M = -INFINITY, z = 0.0;
        const int64_t part = static_cast<int64_t>(first_row + tid) * a.slices;
        if (!(a.finished && a.finished[first_row + tid])) {
            for (int s = 0; s < a.slices; ++s) M = fmax(M, static_cast<double>(__ldcg(a.part_max + part + s)));
            for (int s = 0; s < a.slices; ++s) {
                const double ms = __ldcg(a.part_max + part + s);
                if (ms > -INFINITY) z += __ldcg(a.part_sum + part + s) * exp(ms - M);
            }
        }
        lse[tid] = M > -INFINITY ? M + log(z) : INFINITY;
    }
    if (tid == 0) count = 0;
    __syncthreads();
    // key of list l's entry k (0: none): the score's order; *index its place in beams x vocabulary
    auto entry = [&](int l, int k, int *index) -> uint64_t {
        const int w = l / a.slices;
        const double cum = a.cum[first_row + w];
        double score;
        if (a.finished && a.finished[first_row + w]) {  // its one continuation
            if (l % a.slices || k) return 0;
            *index = w * a.vocab + a.eos;
            score = cum;
        } else {
            const int2 c = __ldcg(reinterpret_cast<const int2 *>(
                a.part_list + (static_cast<int64_t>(first_row) * a.slices + l) * K + k));
            if (c.y < 0) return 0;
            *index = w * a.vocab + c.y;
            score = cum + (static_cast<double>(__int_as_float(c.x)) - lse[w]);
        }
        return score > -INFINITY ? order_key(score) : 0;  // (not -inf, not NaN)
    };
    const int lists = a.beams * a.slices;
    int *join_index = reinterpret_cast<int *>(join_keys + lists * K);
    // The K-th largest list head bounds the K-th best score from below.
    uint64_t least = 1;
    if (lists > K) {
        for (int l = tid; l < lists; l += kThreads) join_keys[l] = entry(l, 0, join_index + l);
        __syncthreads();
        __shared__ uint64_t bound;
        if (tid == 0) bound = 1;
        __syncthreads();
        for (int l = tid; l < lists; l += kThreads) {
            const uint64_t k = join_keys[l];
            int place = 0;
            for (int j = 0; j < lists; ++j) place += join_keys[j] > k || (join_keys[j] == k && j < l);
            if (place == K - 1 && k) bound = k;
        }
        __syncthreads();
        least = bound;
        __syncthreads();
    }
    for (int i = tid; i < lists * K; i += kThreads) {
        int index;
        const uint64_t k = entry(i / K, i % K, &index);
        if (k >= least) {
            const int at = atomicAdd(&count, 1);
            join_keys[at] = k;
            join_index[at] = index;
        }
    }
    __syncthreads();
    const int n = count;
    const int64_t out = static_cast<int64_t>(group) * K;
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = join_keys[i];
        const int index = join_index[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += join_keys[j] > k || (join_keys[j] == k && join_index[j] < index);
        if (place < K) {
            a.scores[out + place] = static_cast<float>(key_value(k));
            a.tokens[out + place] = index % a.vocab;
            a.parents[out + place] = first_row + index / a.vocab;
        }
    }
    for (int i = n + tid; i < K; i += kThreads) {  // fewer candidates than K
        a.scores[out + i] = -INFINITY;
        a.tokens[out + i] = -1;
        a.parents[out + i] = -1;
    }
}

int elem_size(int32_t type) { return type == PA_LOGITS_BF16 ? 2 : type == PA_LOGITS_F32 ? 4 : 0; }

// Slices of a row: enough CTAs to fill the GPU several times over, each with
// at least two vectors per thread, and no more lists than the join holds.
int slices_of(int64_t rows, int beams, int vocab, int K, int elem) {
    const int64_t vecs = (static_cast<int64_t>(vocab) * elem + 15) / 16;
    int64_t s = std::min((vecs + kMinSliceVecs - 1) / kMinSliceVecs, (kTargetCtas + rows - 1) / rows);
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
    const int64_t rows = static_cast<int64_t>(groups) * beams;
    const size_t parts = static_cast<size_t>(rows) * pa::slices_of(rows, beams, vocab, K, pa::elem_size(logits_type));
    return pa::up(4 * static_cast<size_t>(groups)) + pa::up(4 * parts) + pa::up(8 * parts) + pa::up(8 * parts * K);
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
    const int64_t rows = static_cast<int64_t>(groups) * beams;
    pa::BeamArgs a{};
    a.scores = scores, a.tokens = tokens, a.parents = parents;
    a.logits = logits, a.row_stride = row_stride, a.cum = cum, a.finished = finished, a.eos = eos;
    a.beams = beams, a.vocab = vocab, a.K = K;
    a.slices = pa::slices_of(rows, beams, vocab, K, pa::elem_size(logits_type));
    const size_t parts = static_cast<size_t>(rows) * a.slices;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.tickets = reinterpret_cast<int32_t *>(ws);
    ws += pa::up(4 * static_cast<size_t>(groups));
    a.part_max = reinterpret_cast<float *>(ws);
    ws += pa::up(4 * parts);
    a.part_sum = reinterpret_cast<double *>(ws);
    ws += pa::up(8 * parts);
    a.part_list = reinterpret_cast<pa::Candidate *>(ws);
    const int smem = beams * a.slices * K * 12;
    auto kern = logits_type == PA_LOGITS_BF16 ? pa::beam_select_kernel<__nv_bfloat16> : pa::beam_select_kernel<float>;
    static std::atomic<uint64_t> smem_attr_done[2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(smem_attr_done[logits_type].load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, pa::kMaxJoin * 12) != cudaSuccess)
            return PA_ECUDA;
        smem_attr_done[logits_type].fetch_or(bit, std::memory_order_release);
    }
    const cudaError_t e = pa::launch_maybe_cooperative(kern, dim3(static_cast<unsigned>(parts)), pa::kThreads, smem,
                                                       stream, false, pa::pdl_on(), a);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // extern "C"
