// pa_rope.cu -- rotary positions of new queries and keys, and the write of keys
// and values into their cache slots, in one pass.
//
// Pair (a, b) of a head at angle t = pos * freq becomes mscale * (a cos t -
// b sin t, b cos t + a sin t).
//
// Angles.  A frequency becomes a fraction of a turn in 64-bit fixed point, freq / 2 pi mod 1 times
// 2^64 (three fp64 operations per pair and CTA, exact to the frequency's own 53 bits); then
// pos * fraction mod 2^64 is the turn at that position with no rounding at all, for any
// 32-bit position and sign, by one integer multiply -- fp64 arithmetic per (token, pair)
// would cost more than the rotation here.  Its top 32 bits as a signed fraction of a turn feed
// sincospif, whose error and the fp32 rounding are all that is left (about 2^-22).
//
// Work: a CTA puts the R / 2 (cos, sin) pairs of its tokens into shared memory once and
// its threads walk the heads in 16-byte units: a pair of units R / 2 apart, one unit of
// neighbouring pairs, or units behind R, which are copied, as are the values.  Rotary
// dims whose halves are not whole units take the element kernel.
//
// Bound: HBM for a prompt (each q, k, v element read and written once), latency for a step.
#include <cmath>

#include "pa_device.cuh"
#include "pa_scored.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 1024;

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// freq / 2 pi mod 1 in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_fraction(double freq) {
    const double t = freq * 0.15915494309189535;  // 1 / (2 pi)
    return (unsigned long long)((t - floor(t)) * 0x1p64);  // the conversion saturates at 2^64 - 1
}

// (cos, sin) of pos steps of that fraction, times mscale.
__device__ __forceinline__ float2 turn_at(unsigned long long fraction, int pos, float mscale) {
    const int t = (int)((fraction * (unsigned long long)(long long)pos) >> 32);  // turns mod 1, signed, in 2^-32
    float s, c;
    sincospif((float)t * 0x1p-31f, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

// The slot of a token, or -1 for padding; slots past the cache are flagged by one CTA.
__device__ __forceinline__ int64_t token_slot(const RopeArgs &a, int t, bool flag) {
    const int64_t slot = a.slots[t];
    if (slot < 0) return -1;
    if (slot >= (int64_t)a.N * a.B) {
        if (flag) set_error(a.err, PA_DEVERR_BAD_SLOT);
        return -1;
    }
    return slot;
}

// One CTA per token, an element at a time: any even rotary dim.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_elements_kernel(const RopeArgs a) {
    __shared__ float2 cs[kMaxPairs];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x;
    const int64_t slot = token_slot(a, t, threadIdx.x == 0);
    if (slot < 0) return;
    const int half = a.R / 2, pos = a.positions[t];
    for (int i = threadIdx.x; i < half; i += blockDim.x) cs[i] = turn_at(turn_fraction(a.freqs[i]), pos, a.mscale);
    __syncthreads();
    const int64_t blk = slot / a.B, off = slot % a.B;
    const int units = a.D - half;  // per head: R / 2 pairs, then D - R single elements
    for (int u = threadIdx.x; u < (a.Hq + a.Hkv) * units; u += blockDim.x) {
        const int h = u / units, i = u % units;
        const bool is_k = h >= a.Hq;
        const T *src = is_k ? static_cast<const T *>(a.k) + (size_t)t * a.k_stride + (size_t)(h - a.Hq) * a.D
                            : static_cast<const T *>(a.q) + (size_t)t * a.q_stride + (size_t)h * a.D;
        T *dst = is_k ? static_cast<T *>(a.k_cache) + (((size_t)blk * a.Hkv + (h - a.Hq)) * a.B + off) * a.D
                      : static_cast<T *>(a.q_out) + (size_t)t * a.q_out_stride + (size_t)h * a.D;
        if (i < half) {
            const int ia = a.interleaved ? 2 * i : i, ib = a.interleaved ? 2 * i + 1 : i + half;
            const float x = static_cast<float>(src[ia]), y = static_cast<float>(src[ib]);
            const float2 w = cs[i];
            dst[ia] = narrow<T>(x * w.x - y * w.y);
            dst[ib] = narrow<T>(y * w.x + x * w.y);
        } else {
            dst[half + i] = src[half + i];
        }
    }
    for (int u = threadIdx.x; u < a.Hkv * a.D; u += blockDim.x) {
        const int h = u / a.D, d = u % a.D;
        static_cast<T *>(a.v_cache)[(((size_t)blk * a.Hkv + h) * a.B + off) * a.D + d] =
            static_cast<const T *>(a.v)[(size_t)t * a.v_stride + u];
    }
}

template <typename T>
struct alignas(16) Unit {  // 16 bytes of elements
    static constexpr int kN = 16 / sizeof(T);
    T e[kN];
};

// Vector kernel.  grid: (groups of up to kTokens tokens, parts of their heads).  A head is `upq`
// columns: column i holds one unit (interleaved) or two (half layout): the units R / 2 apart
// that rotate together, then pairs of the units behind R.  The heads of q, k and v are numbered
// through and token by token; part y of gridDim.y takes every gridDim.y-th group of them, kU a
// thread in flight.  A thread stays with one column, so its offsets are fixed.
constexpr int kTokens = 4;

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_units_kernel(const RopeArgs a, int tokens, int upq) {
    using U = Unit<T>;
    constexpr int V = U::kN;
    constexpr int kAngles = kInterleaved ? V / 2 : V;  // (cos, sin) pairs of a column
    constexpr int kU = 4;
    extern __shared__ float2 cs[];  // [tokens][R / 2]
    __shared__ int64_t slots[kTokens];
    const int half = a.R / 2, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
    if (tid < nt) slots[tid] = token_slot(a, t0 + tid, blockIdx.y == 0);
    for (int e = tid; e < nt * half; e += kRopeThreads) {
        const int t = e / half, p = e - t * half;
        cs[e] = turn_at(turn_fraction(a.freqs[p]), a.positions[t0 + t], a.mscale);
    }
    __syncthreads();
    const int i = tid % upq, per = kRopeThreads / upq, h0 = tid / upq;
    if (h0 >= per) return;
    const int turning = kInterleaved ? a.R / V : half / V;  // columns that rotate
    const bool turns = i < turning;
    // elements of the column's unit, and from there to its second one
    const int first = kInterleaved || turns ? i * V : a.R + (i - turning) * V;
    const int behind = (a.D - a.R) / V;                     // units behind R, the first half of them paired with the rest
    const int delta = kInterleaved ? 0 : turns ? half : (behind + 1) / 2 * V;
    const bool two = !kInterleaved && (turns || first + delta < a.D);
    const int heads = a.Hq + 2 * a.Hkv, total = nt * heads;
    const int step = per * (int)gridDim.y;
    for (int x0 = blockIdx.y * per + h0; x0 < total; x0 += kU * step) {
        U x[kU], y[kU];
        T *to[kU];
        int tok[kU];  // the token whose angles apply, or -1: a value head
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int n = x0 + u * step;
            const int t = (n >= heads) + (n >= 2 * heads) + (n >= 3 * heads);
            const int h = n - t * heads;
            to[u] = nullptr;
            if (n >= total) continue;
            const int64_t slot = slots[t];
            if (slot < 0) continue;
            const size_t row = t0 + t;
            const int64_t blk = slot / a.B, off = slot - blk * a.B;
            const T *from;
            if (h < a.Hq) {
                from = static_cast<const T *>(a.q) + row * a.q_stride + (size_t)h * a.D;
                to[u] = static_cast<T *>(a.q_out) + row * a.q_out_stride + (size_t)h * a.D;
            } else {
                const bool is_v = h >= a.Hq + a.Hkv;
                const int kh = h - a.Hq - (is_v ? a.Hkv : 0);
                from = static_cast<const T *>(is_v ? a.v : a.k) + row * (is_v ? a.v_stride : a.k_stride) + (size_t)kh * a.D;
                to[u] = static_cast<T *>(is_v ? a.v_cache : a.k_cache) + (((size_t)blk * a.Hkv + kh) * a.B + off) * a.D;
            }
            tok[u] = turns && h < a.Hq + a.Hkv ? t : -1;
            to[u] += first;
            x[u] = *reinterpret_cast<const U *>(from + first);
            if (two) y[u] = *reinterpret_cast<const U *>(from + first + delta);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (!to[u]) continue;
            if (tok[u] >= 0) {
                const float2 *w = cs + tok[u] * half + i * kAngles;
#pragma unroll
                for (int e = 0; e < kAngles; ++e) {
                    T &p = kInterleaved ? x[u].e[2 * e] : x[u].e[e];
                    T &r = kInterleaved ? x[u].e[2 * e + 1] : y[u].e[e];
                    const float pf = static_cast<float>(p), rf = static_cast<float>(r);
                    const float2 c = w[e];
                    p = narrow<T>(pf * c.x - rf * c.y);
                    r = narrow<T>(rf * c.x + pf * c.y);
                }
            }
            *reinterpret_cast<U *>(to[u]) = x[u];
            if (two) *reinterpret_cast<U *>(to[u] + delta) = y[u];
        }
    }
}

template <typename... Args>
cudaError_t launch_rope(void (*kernel)(Args...), dim3 grid, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs &a, cudaStream_t st) {
    constexpr int V = Unit<T>::kN;
    const bool whole = a.interleaved ? a.R % V == 0 : a.R % (2 * V) == 0;
    const int upq = a.interleaved ? a.D / V : a.R / 2 / V + ((a.D - a.R) / V + 1) / 2;
    if (!whole || upq > kRopeThreads) return launch_rope(rope_elements_kernel<T>, dim3((unsigned)a.T), 0, st, a);
    // Few tokens: their heads over several CTAs, down to one head a thread, so that a step's loads are
    // all in flight at once.  Many: four tokens a CTA, whose slots, positions and angles then cost
    // one chain of loads and one barrier.
    const int tokens = a.T >= 16 * 152 && a.R <= 1024 ? kTokens : 1;
    const int groups = (a.T + tokens - 1) / tokens, per = kRopeThreads / upq;
    const int passes = (tokens * (a.Hq + 2 * a.Hkv) + per - 1) / per;
    int parts = (4 * 152 + groups - 1) / groups;
    parts = parts < passes ? parts : passes;
    const dim3 grid((unsigned)groups, (unsigned)(parts > 0 ? parts : 1));
    const size_t smem = (size_t)tokens * (a.R / 2) * sizeof(float2);
    return a.interleaved ? launch_rope(rope_units_kernel<T, true>, grid, smem, st, a, tokens, upq)
                         : launch_rope(rope_units_kernel<T, false>, grid, smem, st, a, tokens, upq);
}

}  // namespace

cudaError_t launch_rope_write_kv(const RopeArgs &a, int dtype, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    if (a.R / 2 > kMaxPairs) return cudaErrorNotSupported;
    if (dtype == PA_F32) return launch_rope_t<float>(a, st);
    if (dtype == PA_F16) return launch_rope_t<__half>(a, st);
    return launch_rope_t<__nv_bfloat16>(a, st);
}

}  // namespace pa
