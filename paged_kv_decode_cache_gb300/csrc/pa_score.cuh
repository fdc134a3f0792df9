// Score rules of pa_decode_scored, shared by the three attention kernels
// (template parameter SC): scores capped by a tanh, a bias that grows with
// distance, a sliding window and a prefix that every query sees.
//
// The tokens that a CTA's queries see are [0, prefix) and [start, stop).  Its
// partitions are counted over VIRTUAL tokens, in which the whole tiles between
// the two are left out, so that unseen blocks are neither loaded nor looked up:
//   real(t) = t for t < head, t + skip from there on
// with head = prefix rounded up to a tile and head + skip = start rounded down
// to one.  Both are multiples of a tile, so a tile of virtual tokens is a tile
// of real ones.  Inside the kept tiles a token is checked by its real place.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

struct Seen {
    int prefix;   // tokens below it are seen by every query
    int start;    // first token in the window of the first query
    int stop;     // past the last query's own position (0: none)
    int head;     // virtual tokens before the gap
    int skip;     // tokens left out
    int end;      // virtual tokens

    __device__ __forceinline__ int real(int t) const { return t < head ? t : t + skip; }
    // whether some query of the CTA sees the (real) token
    __device__ __forceinline__ bool any(int t) const { return t < prefix || (t >= start && t < stop); }
};

// What the queries at positions qbase .. qbase + nq - 1 of a sequence of length
// L (already checked) see.
__device__ __forceinline__ Seen seen_by(const DecodeParams &p, int b, int L, int qbase, int nq, bool report) {
    Seen s;
    s.prefix = 0;
    if (p.prefix_lens) {
        const int n = *reinterpret_cast<const volatile int32_t *>(p.prefix_lens + b);
        if (report && (n < 0 || n > p.max_prefix)) set_status(p.status, PA_STATUS_BAD_SEQLEN);
        s.prefix = min(max(n, 0), min(p.max_prefix, L));
    }
    s.stop = max(0, min(L, qbase + nq));
    s.start = p.window > 0 ? max(0, qbase - p.window + 1) : 0;
    s.head = (s.prefix + kTile - 1) / kTile * kTile;
    s.skip = max(0, s.start / kTile * kTile - s.head);
    s.end = max(s.stop, s.prefix);
    s.end -= s.end > s.head ? s.skip : 0;
    return s;
}

// c tanh(x / c) in log2 units: x and cap are times log2(e), inv_cap = 1 / cap.
// Below u = 0.625 an odd polynomial (a least-squares fit of tanh(u) / u in u^2,
// weighted towards its largest error: 6e-8 of the value in fp32), above 1 - 2 / (e^2u + 1).  Most
// scores are small next to the cap; a warp whose scores all are skips the rest.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], float inv_cap, float cap) {
    bool big = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] *= inv_cap;
        big |= !(fabsf(x[i]) < 0.625f);
    }
    if (!__any_sync(0xffffffffu, big)) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = x[i] * x[i];
            float p = fmaf(t, -0x1.72ef1ep-8f, 0x1.515ceep-6f);
            p = fmaf(t, p, -0x1.b81542p-5f);
            p = fmaf(t, p, 0x1.11058p-3f);
            p = fmaf(t, p, -0x1.555524p-2f);
            x[i] = cap * fmaf(x[i] * t, p, x[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float u = x[i], t = u * u, a = fabsf(u);
        float p = fmaf(t, -0x1.72ef1ep-8f, 0x1.515ceep-6f);
        p = fmaf(t, p, -0x1.b81542p-5f);
        p = fmaf(t, p, 0x1.11058p-3f);
        p = fmaf(t, p, -0x1.555524p-2f);
        const float near = fmaf(u * t, p, u);
        const float far = copysignf(1.f - __fdividef(2.f, fast_exp2(a * 2.8853900817779268f) + 1.f), u);
        x[i] = cap * (a < 0.625f ? near : far);
    }
}

}  // namespace pa
