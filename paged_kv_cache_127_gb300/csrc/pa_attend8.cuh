// pa_attend8.cuh -- what the attention kernels over the 8-bit cache share: which
// keys a sequence's rows see, and the conversions of e4m3 codes.
//
// For the query row at position pos and the keys j with j <= pos and, under a window, j > pos - window or
// j < sinks, with codes k8, v8 and the scales ks, vs of j's block and KV head:
//
//     z_j = scale ks q . k8_j,   out = sum_j p_j vs v8_j,  p = softmax(z).
//
// The scales leave the inner products: with a_j = z_j log2(e) + log2(vs) and m >= all a_j (up to a lag),
// the weights that go into the second product are P_j = 2^(a_j - m) = p_j vs up to a factor, and the
// normaliser is sum_j P_j / vs.  So a scale costs one multiply-add per block and row, the products run on the bare
// codes, and P stays within a bound of its own whatever the blocks' scales are.  Both products take 16-bit floats: an
// e4m3 code is exactly an f16 value (and a bf16 one).  P goes in as two f16 terms (22 bits) where a KV head has at most 16
// rows, as decodes have: HBM bounds those, and the second term costs them little (32 long sequences 207 -> 209 us, a
// batch of 256 79 -> 79, 3 short ones 5.8 -> 6.0).  For more rows P is rounded to f16 once (2^-11 of a weight, where a
// code is off by up to 2^-4 of its value): a second term takes five drafted tokens of 256 sequences from 145 to
// 161 us, 16 x 512-token chunks from 221 to 277 and windowed ones of D 64 from 44 to 54.
// On the tcgen05 path K goes in in the queries' type; on the mma.sync path bf16 queries go in as f16, by a power of two
// per row that brings the row's largest to 2^10, which is exact for every element that is within 2^-24 of it.
#pragma once

#include "pa_device.cuh"
#include "pa_kv8.h"
#include "pa_mma.cuh"

namespace pa {

constexpr float kLog2e8 = 1.4426950408889634f;
constexpr int kStep8 = 32;          // keys of a step of the mma.sync path
constexpr int kStepU8 = 64;         // and of the tcgen05 path
// The largest weights are 2^7 (2^15 with the maximum's lag of 2^8): f16 then keeps 2^-32 of them.
constexpr float kLift8 = 7.f;

// Two e4m3 codes (low byte first) as two f16.
__device__ __forceinline__ uint32_t f16_of_codes(uint32_t lo16) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)lo16));
    return h;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A sequence's part in the call.
struct Seq8 {
    int len, n, q0;  // keys, query rows (tokens), its first row; n 0: nothing to do
};
// `flag`: whether to report what is wrong with it (one thread of the grid does).
__device__ __forceinline__ Seq8 seq_of(const Attend8Args &a, int s, bool flag) {
    Seq8 r;
    r.len = a.context_lens[s];
    const int cap = a.max_blocks * a.B;
    if (r.len < 0 || r.len > cap) {
        if (flag) set_error(a.err, PA_DEVERR_BAD_LEN);
        r.len = r.len < 0 ? 0 : cap;
    }
    r.n = 1;
    r.q0 = s;
    if (a.query_start) {
        r.q0 = a.query_start[s];
        r.n = a.query_start[s + 1] - r.q0;
        if (a.context_lens[s] != r.len || r.n > r.len || r.n > a.max_query_len) {
            if (flag) set_error(a.err, PA_DEVERR_BAD_LEN);
            r.n = 0;
        }
    }
    return r;
}
// Whether query_start is what it has to be at sequence s (a decode has none).
__device__ __forceinline__ bool order_ok(const Attend8Args &a, int s) {
    if (!a.query_start) return true;
    const int b = a.query_start[s], e = a.query_start[s + 1];
    return b >= 0 && e >= b && e <= a.T;
}

// The steps of `keys` keys that rows t0 .. of a sequence walk up to its key `end`: first those that hold sinks,
// then those from the first row's window on.  Step v holds the keys from (v < ns ? v : v + gap) * keys on.
struct Steps8 {
    int ns, gap, count;
};
__device__ __forceinline__ Steps8 steps_of(const Attend8Args &a, int first_pos, int end, int keys) {
    Steps8 r;
    const int begin = a.window > 0 ? max(0, first_pos - a.window + 1) : 0;
    const int b = begin / keys, e = (end + keys - 1) / keys;
    r.ns = min(b, (min(a.sinks, begin) + keys - 1) / keys);
    r.gap = b - r.ns;
    r.count = max(0, e - r.gap);
    return r;
}

// tcgen05 path: the keys [lo, hi) (and sinks) that rows r0 .. r0 + 128 a.tiles - 1 of a sequence see, and their steps.
struct Span8 {
    int lo, hi;
    Steps8 st;
};
__device__ __forceinline__ Span8 span_of(const Attend8Args &a, const Seq8 &q, int r0) {
    const int G = a.Hq / a.Hkv, first = q.len - q.n + r0 / G;
    Span8 r;
    r.hi = q.len - q.n + min(q.n - 1, (r0 + 128 * a.tiles - 1) / G) + 1;
    r.lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
    r.st = steps_of(a, first, r.hi, kStepU8);
    return r;
}

}  // namespace pa
