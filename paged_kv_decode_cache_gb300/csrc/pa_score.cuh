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
// With u = x / cap below 0.625, x (1 + u^2 p(u^2)) with a least-squares fit of
// tanh(u) / u weighted towards its largest error: 6e-8 of the value in fp32.  From
// there on 1 - 2 / (e^2u + 1), whose error is 2^-22 of the cap.  Each score takes the
// form of its own size, so that its bits depend on it alone: a warp also holds rows
// that no query sees, which may be anything.  The warp's vote only skips the second
// form where no lane needs it (most scores are small next to the cap; 9 operations,
// two scores each).
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], float inv_cap, float cap) {
    bool big = false;
    const float edge = 0.625f * cap;
    const uint64_t ic = pack2(inv_cap, inv_cap);
    auto near = [&](float x0, float x1, float &a, float &b) {
        const uint64_t v = pack2(x0, x1), u = mul2(v, ic), t = mul2(u, u);
        uint64_t p = fma2(t, pack2(-0x1.72ef1ep-8f, -0x1.72ef1ep-8f), pack2(0x1.515ceep-6f, 0x1.515ceep-6f));
        p = fma2(t, p, pack2(-0x1.b81542p-5f, -0x1.b81542p-5f));
        p = fma2(t, p, pack2(0x1.11058p-3f, 0x1.11058p-3f));
        p = fma2(t, p, pack2(-0x1.555524p-2f, -0x1.555524p-2f));
        unpack2(fma2(mul2(v, t), p, v), a, b);
    };
#pragma unroll
    for (int i = 0; i < N; ++i) big |= !(fabsf(x[i]) < edge);
    if (!__any_sync(0xffffffffu, big)) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float a, b;
            near(x[i], x[i + 1 < N ? i + 1 : i], a, b);
            x[i] = a;
            if (i + 1 < N) x[i + 1] = b;
        }
        return;
    }
    const float k = 2.8853900817779268f * inv_cap;  // e^2u = 2^(k x)
    auto pick = [&](float v, float small) {
        const float far = fmaf(-cap, __fdividef(2.f, fast_exp2(fabsf(v) * k) + 1.f), cap);
        return fabsf(v) < edge ? small : copysignf(far, v);
    };
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float a, b;
        near(x[i], x[i + 1 < N ? i + 1 : i], a, b);
        x[i] = pick(x[i], a);
        if (i + 1 < N) x[i + 1] = pick(x[i + 1], b);
    }
}

}  // namespace pa
