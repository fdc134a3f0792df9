// Rotary positions fused with the slot-mapping cache write: one launch turns a
// step's query heads and new key heads and writes K and V into the pools.
//
// Pair (a, b) of a head at position p turns by t = p f: a' = m (a cos t - b sin t),
// b' = m (a sin t + b cos t).  The plan holds f / 2 pi as a 64-bit fraction of a turn;
// p times it modulo 2^64 is exact, so that the angle is off by the plan's own rounding,
// about p 2^-54 turns; its top 32 bits, as a signed number of half turns, go to
// sincospi.  (p f in fp32 is off by p 2^-25 radians: 0.03 at a million.)
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kUnit = 16;          // elements per thread: 8 pairs, two 16-byte chunks
constexpr int kMaxThreads = 512;

struct RopeArgs {
    __nv_bfloat16 *q_out;
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_out_stride, q_stride, k_stride, v_stride;
    const int32_t *positions;
    const int64_t *slots;
    int64_t n, n_slots;
    uint8_t *k_cache, *v_cache;
    int32_t *status;
    int hq, hkv, head_dim;
    float k_scale, v_scale;        // FP8 pools
    float k_inv, v_inv;            // their reciprocals (e4m3x8_from_f32)
};

// Thread = one unit of 16 elements of one head of q, k or v, for groups of TB
// tokens: two 16-byte chunks half of the turning dimensions apart (of the others
// where nothing turns), which holds 8 whole pairs in either layout.  Neighbouring
// threads take neighbouring chunks, so that a warp reads and writes whole lines.
// A CTA's groups are gridDim.x apart: while one is turned, the next one's angles are
// computed (one per thread at a time, kept in shared memory for all heads) from
// positions read a group earlier, and a thread's loads run a token ahead, across
// groups (two tokens ahead 45.3 us, four 50.8; with 1280 threads per SM 48.2, with
// 768 49.3: 16384 tokens of 32 heads into FP8 pools).
// Bound by a launch for a decode step (8 tokens of 36 heads: 2.3 us), by memory for
// prompts (those 16384 tokens 41.2 us, 0.85 of the copy rate, into bf16 pools 43, 0.92).
template <bool F8, int TB, bool HALF>
__global__ void __launch_bounds__(kMaxThreads, 2)
rope_write_kernel(const RopeArgs a, const __grid_constant__ pa_rope rope) {
    __shared__ __align__(16) float2 turn[2][TB][PA_ROPE_MAX_PAIRS];  // (cos, sin) of the pairs: this group's, the next one's
    __shared__ int32_t pos_s[2][TB];                             // positions of the next two groups
    __shared__ int64_t row_s[3][TB];                             // rows in the pools, in elements (-1: not written)
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * TB;   // a CTA's groups, in tokens
    const int units = a.head_dim / kUnit, rot_units = rope.rot_dim / kUnit, pairs = rope.rot_dim / 2;
    const int total = (a.hq + 2 * a.hkv) * units, x = blockIdx.y * blockDim.x + tid;
    const int head = min(x, total - 1) / units, u = x % units;
    const bool is_q = head < a.hq, is_v = head >= a.hq + a.hkv;
    const bool rotates = u < rot_units && !is_v;
    // its two chunks: half of the dimensions that turn, or of the others, apart
    const int from = rotates || is_v ? 0 : rope.rot_dim;
    const int apart = (rotates ? rope.rot_dim : a.head_dim - from) / 2;
    const int e0 = from + 8 * (from ? u - rot_units : u);
    const int at_head = (head - (is_q ? 0 : is_v ? a.hq + a.hkv : a.hq)) * a.head_dim + e0;
    const int64_t stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
    const __nv_bfloat16 *src = (is_q ? a.q : is_v ? a.v : a.k) + at_head;
    uint4 lo, hi;
    auto load = [&](int64_t tok) {
        lo = hi = make_uint4(0u, 0u, 0u, 0u);
        if (tok < a.n && x < total) {
            lo = *reinterpret_cast<const uint4 *>(src + tok * stride);
            hi = *reinterpret_cast<const uint4 *>(src + tok * stride + apart);
        }
    };
    auto row_of = [&](int64_t tok) -> int64_t {
        const int64_t slot = a.slots[tok];
        if (slot >= a.n_slots) set_status(a.status, PA_STATUS_BAD_SLOT);
        return slot < 0 || slot >= a.n_slots ? -1 : slot * a.hkv * a.head_dim;
    };
    auto angles = [&](int buf, int tokens, auto &&position) {
        for (int i = tid; i < tokens * pairs; i += blockDim.x) {
            const int at = i / pairs, k = i % pairs;
            const uint64_t f = static_cast<uint64_t>(static_cast<int64_t>(position(at))) * rope.turn[k];
            float s, c;
            sincospif(static_cast<float>(static_cast<int32_t>(f >> 32)) * 0x1p-31f, &s, &c);
            turn[buf][at][k] = make_float2(c * rope.magnitude, s * rope.magnitude);
        }
    };
    auto tokens_from = [&](int64_t tok) { return static_cast<int>(min(static_cast<int64_t>(TB), a.n - tok)); };

    int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TB;
    load(tok0);
    angles(0, tokens_from(tok0), [&](int at) { return a.positions[tok0 + at]; });
    if (tid < TB && tok0 + tid < a.n) row_s[0][tid] = row_of(tok0 + tid);
    if (tid < TB && tok0 + step + tid < a.n) {
        pos_s[1][tid] = a.positions[tok0 + step + tid];
        row_s[1][tid] = row_of(tok0 + step + tid);
    }
    __syncthreads();
    for (int buf = 0, row3 = 0;; buf ^= 1, row3 = row3 == 2 ? 0 : row3 + 1, tok0 += step) {
        const bool more = tok0 + step < a.n, mine = tid < TB && tok0 + 2 * step + tid < a.n;
        int32_t pos2 = 0;
        int64_t row2 = -1;
        if (mine) pos2 = a.positions[tok0 + 2 * step + tid], row2 = row_of(tok0 + 2 * step + tid);
        if (more) angles(buf ^ 1, tokens_from(tok0 + step), [&](int at) { return pos_s[buf ^ 1][at]; });
        const int tokens = tokens_from(tok0);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const uint4 now_lo = lo, now_hi = hi;
            // (in place too: another token than the one written below)
            if (TB > 1) load(t + 1 < TB ? tok0 + t + 1 : tok0 + step);
            if (t >= tokens || x >= total) continue;
            const int64_t row = row_s[row3][t];
            if (!is_q && row < 0) continue;
            const uint32_t w0[4] = {now_lo.x, now_lo.y, now_lo.z, now_lo.w};
            const uint32_t w1[4] = {now_hi.x, now_hi.y, now_hi.z, now_hi.w};
            float f0[8], f1[8];  // the two chunks' values
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f0[2 * i] = bf16lo(w0[i]), f0[2 * i + 1] = bf16hi(w0[i]);
                f1[2 * i] = bf16lo(w1[i]), f1[2 * i + 1] = bf16hi(w1[i]);
            }
            if (rotates) {
                // pairs 8 u .. 8 u + 7, one of each in either chunk (half), or 4 u .. 4 u + 3 in
                // the first and as many, rot_dim / 4 on, in the second (interleaved)
                const float2 *turns = turn[buf][t];
                const float4 *c0 = reinterpret_cast<const float4 *>(turns + (HALF ? 8 * u : 4 * u));
                const float4 *c1 = HALF ? c0 + 2 : reinterpret_cast<const float4 *>(turns + rope.rot_dim / 4 + 4 * u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 two = i < 4 ? c0[i / 2] : c1[i / 2 - 2];
                    const float c = i & 1 ? two.z : two.x, s = i & 1 ? two.w : two.y;
                    float *fa = HALF ? f0 + i : i < 4 ? f0 + 2 * i : f1 + 2 * i - 8;
                    float *fb = HALF ? f1 + i : fa + 1;
                    const float x0 = *fa, x1 = *fb;
                    *fa = x0 * c - x1 * s;
                    *fb = x0 * s + x1 * c;
                }
            }
            if (F8 && !is_q) {
                const float scale = is_v ? a.v_scale : a.k_scale, inv = is_v ? a.v_inv : a.k_inv;
                uint8_t *dst = (is_v ? a.v_cache : a.k_cache) + row + at_head;
                *reinterpret_cast<uint2 *>(dst) = e4m3x8_from_f32(f0, scale, inv);
                *reinterpret_cast<uint2 *>(dst + apart) = e4m3x8_from_f32(f1, scale, inv);
            } else {
                __nv_bfloat16 *dst = is_q ? a.q_out + (tok0 + t) * a.q_out_stride + at_head
                                          : reinterpret_cast<__nv_bfloat16 *>(is_v ? a.v_cache : a.k_cache) + row + at_head;
                uint32_t o0[4], o1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b0 = __floats2bfloat162_rn(f0[2 * i], f0[2 * i + 1]);
                    const __nv_bfloat162 b1 = __floats2bfloat162_rn(f1[2 * i], f1[2 * i + 1]);
                    o0[i] = rotates ? *reinterpret_cast<const uint32_t *>(&b0) : w0[i];  // (a copy keeps its bits)
                    o1[i] = rotates ? *reinterpret_cast<const uint32_t *>(&b1) : w1[i];
                }
                *reinterpret_cast<uint4 *>(dst) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
                *reinterpret_cast<uint4 *>(dst + apart) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            }
        }
        if (!more) break;
        if (mine) pos_s[buf][tid] = pos2, row_s[row3 == 0 ? 2 : row3 - 1][tid] = row2;
        __syncthreads();
    }
}

float reciprocal(float scale) { return scale > 0x1p-60f && scale < 0x1p60f ? 1.f / scale : NAN; }

// Tokens per group: one, and a CTA for each, where there are few (600 tokens of 32 heads
// into FP8 pools: 3.4 us, with four 4.3); else four (1536 tokens of 36 heads: 6.3 us,
// with one 8.9), and as many CTAs as the GPU holds at once.
constexpr int kFourFrom = 768;

template <bool F8, int TB>
cudaError_t launch_rope_instance(const RopeArgs &a, const pa_rope &rope, cudaStream_t stream) {
    const int units = (a.hq + 2 * a.hkv) * (a.head_dim / kUnit), parts = (units + kMaxThreads - 1) / kMaxThreads;
    const int threads = ((units + parts - 1) / parts + 31) / 32 * 32;
    int64_t ctas = (a.n + TB - 1) / TB;
    if (TB > 1) ctas = std::min<int64_t>(ctas, std::max(1, sm_count() * std::max(1, kMaxThreads * 2 / threads) / parts));
    return launch_maybe_cooperative(rope.layout == PA_ROPE_HALF ? rope_write_kernel<F8, TB, true>
                                                                : rope_write_kernel<F8, TB, false>,
                                    dim3(static_cast<unsigned>(ctas), parts), threads, 0, stream, false, pdl_on(), a, rope);
}

template <bool F8>
cudaError_t launch_rope(const RopeArgs &a, const pa_rope &rope, cudaStream_t stream) {
    return a.n < kFourFrom ? launch_rope_instance<F8, 1>(a, rope, stream) : launch_rope_instance<F8, 4>(a, rope, stream);
}

int rope_write(bool f8, void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k_new,
               int64_t k_stride, const void *v_new, int64_t v_stride, const int32_t *positions,
               const int64_t *slot_mapping, int64_t n_tokens, int32_t Hq, void *k_cache, void *v_cache,
               const pa_cache_desc &cache, float k_scale, float v_scale, const pa_rope *rope, int32_t *status,
               cudaStream_t stream) {
    if (n_tokens < 0 || Hq <= 0 || !rope) return PA_EINVAL;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (rope->rot_dim <= 0 || rope->rot_dim % kUnit != 0 ||
        (rope->layout != PA_ROPE_HALF && rope->layout != PA_ROPE_INTERLEAVED))
        return PA_EINVAL;
    if (rope->rot_dim > cache.head_dim) return PA_EINVAL;
    if (f8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale)))
        return PA_EINVAL;
    if (n_tokens > INT32_MAX || static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(cache.num_kv_heads) > (1 << 20))
        return PA_EUNSUPPORTED;
    if (n_tokens == 0) return PA_OK;
    if (!q_out || !q || !k_new || !v_new || !positions || !slot_mapping || !k_cache || !v_cache) return PA_EINVAL;
    for (const void *p : {static_cast<const void *>(q_out), q, k_new, v_new, static_cast<const void *>(k_cache),
                          static_cast<const void *>(v_cache)})
        if (!is_aligned(p, 16)) return PA_EINVAL;
    if (!is_aligned(positions, 4) || !is_aligned(slot_mapping, 8)) return PA_EINVAL;
    const int64_t q_row = static_cast<int64_t>(Hq) * cache.head_dim;
    const int64_t kv_row = static_cast<int64_t>(cache.num_kv_heads) * cache.head_dim;
    if (q_out_stride < q_row || q_stride < q_row || k_stride < kv_row || v_stride < kv_row ||
        ((q_out_stride | q_stride | k_stride | v_stride) & 7))
        return PA_EINVAL;
    RopeArgs a{static_cast<__nv_bfloat16 *>(q_out), static_cast<const __nv_bfloat16 *>(q),
               static_cast<const __nv_bfloat16 *>(k_new), static_cast<const __nv_bfloat16 *>(v_new),
               q_out_stride, q_stride, k_stride, v_stride, positions, slot_mapping, n_tokens,
               static_cast<int64_t>(cache.num_blocks) * cache.block_size, static_cast<uint8_t *>(k_cache),
               static_cast<uint8_t *>(v_cache), status, Hq, cache.num_kv_heads, cache.head_dim, k_scale, v_scale, reciprocal(k_scale), reciprocal(v_scale)};
    const cudaError_t e = f8 ? launch_rope<true>(a, *rope, stream) : launch_rope<false>(a, *rope, stream);
    return e == cudaSuccess ? PA_OK : PA_ECUDA;
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_rope_init(pa_rope *rope, int32_t rot_dim, int32_t layout, double base, const pa_rope_scaling *scaling) {
    if (!rope || rot_dim <= 0) return PA_EINVAL;
    if (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED) return PA_EINVAL;
    if (rot_dim % pa::kUnit != 0 || rot_dim > 2 * PA_ROPE_MAX_PAIRS) return PA_EUNSUPPORTED;
    if (!(base > 1.0) || !std::isfinite(base)) return PA_EINVAL;
    const pa_rope_scaling none{PA_ROPE_PLAIN, 1.0, 0.0, 0.0, 0.0, 0.0};
    const pa_rope_scaling &sc = scaling ? *scaling : none;
    const bool by_turns = sc.kind == PA_ROPE_YARN || sc.kind == PA_ROPE_BANDED;
    if (sc.kind < PA_ROPE_PLAIN || sc.kind > PA_ROPE_BANDED) return PA_EINVAL;
    if (sc.kind != PA_ROPE_PLAIN && (!(sc.factor > 0.0) || !std::isfinite(sc.factor))) return PA_EINVAL;
    if (sc.kind == PA_ROPE_YARN && sc.factor < 1.0) return PA_EINVAL;
    if (by_turns && (!(sc.original_positions > 0.0) || !std::isfinite(sc.original_positions) || !(sc.low > 0.0) ||
                     !(sc.high > sc.low) || !std::isfinite(sc.high)))
        return PA_EINVAL;
    if (!(sc.magnitude >= 0.0) || !std::isfinite(sc.magnitude)) return PA_EINVAL;

    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const double b = sc.kind == PA_ROPE_NTK
                         ? base * std::pow(sc.factor, rot_dim / static_cast<double>(rot_dim - 2))
                         : base;
    // YaRN: the (real) pair index whose frequency makes n turns over the original positions
    auto pair_of = [&](double n) {
        return rot_dim * std::log(sc.original_positions / (n * kTwoPi)) / (2.0 * std::log(base));
    };
    double lo = 0.0, hi = 0.0;
    if (sc.kind == PA_ROPE_YARN) {
        lo = std::max(std::floor(pair_of(sc.high)), 0.0);
        hi = std::min(std::ceil(pair_of(sc.low)), static_cast<double>(rot_dim - 1));
    }
    for (int i = 0; i < PA_ROPE_MAX_PAIRS; ++i) {
        rope->turn[i] = 0;
        if (i >= rot_dim / 2) continue;
        double f = std::pow(b, -2.0 * i / rot_dim);
        double slow = 0.0;  // share of the frequency that is divided by the factor
        if (sc.kind == PA_ROPE_LINEAR) slow = 1.0;
        if (sc.kind == PA_ROPE_YARN) slow = std::clamp((i - lo) / std::max(hi - lo, 0.001), 0.0, 1.0);
        if (sc.kind == PA_ROPE_BANDED)
            slow = 1.0 - std::clamp((sc.original_positions * f / kTwoPi - sc.low) / (sc.high - sc.low), 0.0, 1.0);
        if (slow > 0.0) f = f / sc.factor * slow + f * (1.0 - slow);
        double turns = f / kTwoPi;
        turns -= std::floor(turns);  // (a factor below 1 can push it past one turn)
        rope->turn[i] = static_cast<uint64_t>(std::llround(std::ldexp(turns, 62))) << 2;
    }
    rope->magnitude = static_cast<float>(sc.magnitude > 0.0             ? sc.magnitude
                                         : sc.kind == PA_ROPE_YARN ? 0.1 * std::log(sc.factor) + 1.0
                                                                   : 1.0);
    rope->rot_dim = rot_dim;
    rope->layout = layout;
    return PA_OK;
}

int pa_rope_write(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k_new,
                  int64_t k_stride, const void *v_new, int64_t v_stride, const int32_t *positions,
                  const int64_t *slot_mapping, int64_t n_tokens, int32_t Hq, void *k_cache, void *v_cache,
                  pa_cache_desc cache, const pa_rope *rope, int32_t *status, pa_stream_t stream) {
    return pa::rope_write(false, q_out, q_out_stride, q, q_stride, k_new, k_stride, v_new, v_stride, positions,
                          slot_mapping, n_tokens, Hq, k_cache, v_cache, cache, 1.f, 1.f, rope, status, stream);
}

int pa_rope_write_fp8(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k_new,
                      int64_t k_stride, const void *v_new, int64_t v_stride, const int32_t *positions,
                      const int64_t *slot_mapping, int64_t n_tokens, int32_t Hq, void *k_cache, void *v_cache,
                      pa_cache_desc cache, float k_scale, float v_scale, const pa_rope *rope, int32_t *status,
                      pa_stream_t stream) {
    return pa::rope_write(true, q_out, q_out_stride, q, q_stride, k_new, k_stride, v_new, v_stride, positions,
                          slot_mapping, n_tokens, Hq, k_cache, v_cache, cache, k_scale, v_scale, rope, status,
                          stream);
}

}  // extern "C"
