// pa_score.cuh -- device side of pa_score: the range of keys a query row sees
// and the cap and bias of a logit.
#pragma once

#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_scored.h"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr float kLog2e = 1.4426950408889634f;

// How far below a row's largest logit, in log2 units, its softmax takes the maximum that weights are relative
// to.  Two f16 parts keep a weight to 2^-25 at best, so with weights of at most 1 those below 2^-25 of the largest
// would be lost from P V but not from the row's sum (a dominant key and 2^17 others at 2^-26: 0.2 % of the mass).
// Weights of up to 2^15, just inside f16, keep them down to 2^-40 of the largest; the row's sum is in the same units,
// so nothing is divided out.  bf16 has the exponents of fp32 and needs no lift.
template <typename T>
constexpr float kWeightLift = std::is_same<T, __half>::value ? 15.f : 0.f;

// Keys [x, y) that row i, at position pos of a sequence of len tokens, sees;
// (0, 0) when none is left.
__device__ __forceinline__ int2 row_range(const ScoredArgs &a, int i, int pos, int len) {
    int begin = a.key_begin ? max(0, a.key_begin[i]) : 0;
    if (a.window > 0) begin = max(begin, pos - a.window + 1);
    const int end = min(len, a.key_end ? a.key_end[i] : pos + 1);
    return begin < end ? make_int2(begin, end) : make_int2(0, 0);
}

// The pieces in which a listed decode splits a sequence's range [x, y): the first ends at
// the next multiple of the partition size, `size`, the others at multiples of the size that
// the plan chose, `wide` (a multiple of it).  Their number, and piece i.
__device__ __forceinline__ int pieces_of(int2 k, int size, int wide) {
    const int e = (k.x / size + 1) * size;
    return e >= k.y ? 1 : 1 + (k.y - 1) / wide - e / wide + 1;
}
__device__ __forceinline__ int2 piece_of(int2 k, int size, int wide, int i) {
    const int e = (k.x / size + 1) * size;
    if (i == 0) return make_int2(k.x, min(k.y, e));
    const int w = e / wide + i - 1;
    return make_int2(max(e, w * wide), min(k.y, (w + 1) * wide));
}

// The sequence, position and length of query row i: a decode's row is its
// sequence's last token (a length outside [0, cap] is clamped); a chunk's row
// belongs to the last sequence s with query_start[s] <= i.  s = -1 when the row
// has no sequence or its sequence is not worked on.  chunk_ok: query_start is
// non-decreasing within [0, T] (checked once per launch).
struct RowOf {
    int s, pos, len;
};
__device__ __forceinline__ RowOf row_of(const ScoredArgs &a, int i, int cap) {
    RowOf r{-1, 0, 0};
    if (!a.query_start) {
        int len = a.context_lens[i];
        len = len < 0 ? 0 : (len > cap ? cap : len);
        r.s = i, r.pos = len - 1, r.len = len;
        return r;
    }
    int lo = 0, hi = a.S;  // query_start[lo] <= i (or lo == 0), the answer in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.query_start[mid] <= i) lo = mid; else hi = mid;
    }
    const int q0 = a.query_start[lo], q1 = a.query_start[lo + 1];
    if (i < q0 || i >= q1) return r;
    const int n = q1 - q0, len = a.context_lens[lo];
    if (len < 0 || len > cap || n > len || n > a.max_query_len) return r;
    r.s = lo, r.pos = len - n + (i - q0), r.len = len;
    return r;
}

// tanh(y) = y P(y^2) / Q(y^2), both of degree 4, on |y| <= 9, past which tanh
// rounds to 1 in fp32: a least-squares fit of the relative error, reweighted
// towards its maximum until level (2.1e-8), with fp32 coefficients.  Evaluated in fp32 with
// the approximate reciprocal it is within 2^-21 of tanh, relative (rms 2^-24).  NaN stays NaN: fminf and
// fmaxf would return the bound, and a NaN score would pass for one at the cap.
__device__ __forceinline__ float rational_tanh(float y) {
    asm("max.NaN.f32 %0, %0, 0fC1100000;" : "+f"(y));  // -9
    asm("min.NaN.f32 %0, %0, 0f41100000;" : "+f"(y));  // 9
    const float z = y * y;
    float p = fmaf(z, 1.3354597427905901e-08f, 2.060904989775736e-05f);
    p = fmaf(p, z, 0.0034955868031829596f);
    p = fmaf(p, z, 0.13381025195121765f);
    p = fmaf(p, z, 1.f);
    float q = fmaf(z, 7.776536108394794e-07f, 0.0003285632119514048f);
    q = fmaf(q, z, 0.025876978412270546f);
    q = fmaf(q, z, 0.4671434164047241f);
    q = fmaf(q, z, 1.f);
    return __fdividef(y * p, q);
}

// A logit in log2 units from a dot product: scaled, capped.
struct ScoreCap {
    float in, out;  // log2 logit = out * tanh(in * dot) with a cap, else in * dot
    bool cap;
    __device__ __forceinline__ explicit ScoreCap(const ScoredArgs &a) {
        cap = a.softcap > 0.f;
        in = cap ? a.scale / a.softcap : a.scale * kLog2e;
        out = a.softcap * kLog2e;
    }
    __device__ __forceinline__ float operator()(float dot) const {
        return cap ? out * rational_tanh(in * dot) : in * dot;
    }
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The cap on N raw dot products in place, in raw units: f -> tanh(in f) / in, so
// that the logit is f times the plain scale with a cap or without.  Needs in > 0;
// `most` is at least every |f| of the calling thread.  Logits rarely come near their cap, so a
// whole warp mostly takes the first form:
//   |in f| <= 0.5   f + f^3 (c1 + c2 f^2 + c3 f^4 + c4 f^6): tanh(y) = y (1 + y^2 Q(y^2)), Q of
//                   degree 3 (fitted as above, 1.5e-8), the powers of `in` taken into its coefficients;
//   |in f| <= 0.9   y P(y^2), P of degree 6 (1.4e-8);
//   else            the rational form.
// The polynomials cost 3 and 4.5 issue slots a value in packed arithmetic and no
// special function, the rational form 15 and a reciprocal.
struct CapFit {
    float in, c1, c2, c3, c4, near;
    __device__ __forceinline__ explicit CapFit(float in_) : in(in_) {
        const float z = in * in;
        c1 = -0.333331435918808f * z;
        c2 = 0.13325878977775574f * z * z;
        c3 = -0.05304549261927605f * z * z * z;
        c4 = 0.01724148355424404f * z * z * (z * z);
        // the scaled coefficients and the powers of f stay normal numbers in this range of `in`
        near = in >= 0x1p-14f && in <= 0x1p10f ? 0.5f / in : -1.f;
    }
};
// Its first form.
template <int N>
__device__ __forceinline__ void cap_near(float (&f)[N], const CapFit &c) {
    auto both = [](float x) { return tc::f2(x, x); };
    const uint64_t c1 = both(c.c1), c2 = both(c.c2), c3 = both(c.c3), c4 = both(c.c4);
#pragma unroll
    for (int v = 0; v < N / 2; ++v) {
        const uint64_t x = tc::f2(f[2 * v], f[2 * v + 1]);
        const uint64_t z = mul2(x, x);
        const uint64_t q = tc::fma2(tc::fma2(tc::fma2(z, c4, c3), z, c2), z, c1);
        const float2 r = tc::f2split(tc::fma2(mul2(x, z), q, x));
        f[2 * v] = r.x;
        f[2 * v + 1] = r.y;
    }
}
template <int N>
__device__ __forceinline__ void cap_in_place(float (&f)[N], const CapFit &c, float most) {
    auto both = [](float x) { return tc::f2(x, x); };
    if (__all_sync(0xffffffffu, most <= c.near)) {
        cap_near(f, c);
    } else if (__all_sync(0xffffffffu, most * c.in <= 0.9f)) {
        const uint64_t in2 = both(c.in);
#pragma unroll
        for (int v = 0; v < N / 2; ++v) {
            const uint64_t x = tc::f2(f[2 * v], f[2 * v + 1]);
            const uint64_t y = mul2(x, in2), z = mul2(y, y);
            uint64_t p = tc::fma2(z, both(0.001286464394070208f), both(-0.006814091932028532f));
            p = tc::fma2(p, z, both(0.020857738330960274f));
            p = tc::fma2(p, z, both(-0.0536990687251091f));
            p = tc::fma2(p, z, both(0.1332983523607254f));
            p = tc::fma2(p, z, both(-0.3333316147327423f));
            p = tc::fma2(p, z, both(1.f));
            const float2 r = tc::f2split(mul2(x, p));
            f[2 * v] = r.x;
            f[2 * v + 1] = r.y;
        }
    } else {
        const float back = 1.f / c.in;
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = back * rational_tanh(c.in * f[i]);
    }
}

}  // namespace pa
