// pa_score.cuh -- device side of pa_score: the range of keys a query row sees
// and the cap and bias of a logit.
#pragma once

#include <cmath>

#include "pa_device.cuh"
#include "pa_scored.h"

namespace pa {

constexpr float kLog2e = 1.4426950408889634f;

// Keys [x, y) that row i, at position pos of a sequence of len tokens, sees;
// (0, 0) when none is left.
__device__ __forceinline__ int2 row_range(const ScoredArgs &a, int i, int pos, int len) {
    int begin = a.key_begin ? max(0, a.key_begin[i]) : 0;
    if (a.window > 0) begin = max(begin, pos - a.window + 1);
    const int end = min(len, a.key_end ? a.key_end[i] : pos + 1);
    return begin < end ? make_int2(begin, end) : make_int2(0, 0);
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
// the approximate reciprocal it is within 2^-21 of tanh, relative (rms 2^-24).
__device__ __forceinline__ float rational_tanh(float y) {
    y = fminf(fmaxf(y, -9.f), 9.f);
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

// One output value rounded to the output's type.
template <typename T>
__device__ __forceinline__ void store_out(T *p, float x);
template <>
__device__ __forceinline__ void store_out<float>(float *p, float x) { *p = x; }
template <>
__device__ __forceinline__ void store_out<__half>(__half *p, float x) { *p = __float2half_rn(x); }
template <>
__device__ __forceinline__ void store_out<__nv_bfloat16>(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

}  // namespace pa
