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
