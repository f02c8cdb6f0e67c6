// pa_rope.cu -- rotary positions of new queries and keys, and the write of keys
// and values into their cache slots, in one pass.
//
// Pair (a, b) of a head at angle t = pos * freq becomes mscale * (a cos t -
// b sin t, b cos t + a sin t).  With several axes each pair has a position of its own
// (pair_position); everything behind the angles is the same.
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
// neighbouring pairs, or units behind R, which are copied, as are the values.  Where half
// the rotary dim is not whole units (in the half layout), a thread takes one unit and its elements'
// partners one by one (from L1); heads of more than 256 units go element by element.
//
// Bound: HBM for a prompt (each q, k, v element read and written once), latency for a step.
// Measured: 8192 tokens of 32 + 32 heads (D 128, f16, 64 elements rotated as neighbours) 64 us (floor 59), of
// 32 + 8 heads (bf16, whole heads in halves) 37 (floor 30), with three axes 38; the kernel of a step of 256 tokens, 64 + 8
// heads, 4.8 us, of one token 2.8 us.
#include <cmath>

#include "pa_device.cuh"
#include "pa_mma.cuh"
#include "pa_rope.cuh"
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

// One CTA per token, an element at a time: any even rotary dim and head.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_elements_kernel(const RopeArgs a) {
    __shared__ float2 cs[kMaxPairs];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x;
    const int64_t slot = token_slot(a, t, threadIdx.x == 0);
    if (slot < 0) return;
    const int half = a.R / 2;
    for (int i = threadIdx.x; i < half; i += blockDim.x)
        cs[i] = turn_at(turn_fraction(a.freqs[i]), pair_position(a, t, i), a.mscale);
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
            const float2 w = turned(x, y, cs[i]);
            dst[ia] = narrow<T>(w.x);
            dst[ib] = narrow<T>(w.y);
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

// A 16-byte unit of elements, as fp32 and back (each element rounded once).
template <typename T>
struct Unit {
    static constexpr int kN = 16 / sizeof(T);
    static __device__ __forceinline__ uint4 pack(const float *f) {
        if constexpr (sizeof(T) == 4)
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        else
            return make_uint4(Mma16<T>::pack(f[0], f[1]), Mma16<T>::pack(f[2], f[3]), Mma16<T>::pack(f[4], f[5]),
                              Mma16<T>::pack(f[6], f[7]));
    }
};

// Vector kernel.  grid: (groups of up to kTokens tokens, parts of their heads).  A head is `upq`
// columns: column i holds one unit (interleaved) or two (half layout): the units R / 2 apart
// that rotate together, then pairs of the units behind R.  The heads of q, k and v are numbered
// through; part y of gridDim.y takes every gridDim.y-th group of them, kU a thread in flight.
// A thread stays with one column, so its offsets within a head are fixed.
constexpr int kTokens = 2;

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_units_kernel(const RopeArgs a, int tokens, int upq) {
    constexpr int V = Unit<T>::kN;
    constexpr int kAngles = kInterleaved ? V / 2 : V;  // (cos, sin) pairs of a column
    constexpr int kU = kInterleaved ? 6 : 4;
    extern __shared__ float2 cs[];  // [tokens][R / 2]
    __shared__ int64_t slots[kTokens];
    const int half = a.R / 2, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
    if (tid < nt) slots[tid] = token_slot(a, t0 + tid, blockIdx.y == 0);
    for (int e = tid; e < nt * half; e += kRopeThreads) {
        const int t = e / half, p = e - t * half;
        cs[e] = turn_at(turn_fraction(a.freqs[p]), pair_position(a, t0 + t, p), a.mscale);
    }
    __syncthreads();
    const int i = tid % upq, per = kRopeThreads / upq, h0 = tid / upq;
    if (h0 >= per) return;
    const int turning = kInterleaved ? (a.R + V - 1) / V : half / V;  // columns that rotate
    const bool turns = i < turning;
    const int live = kInterleaved ? min(kAngles, half - i * kAngles) : kAngles;  // pairs of the unit that do
    // elements of the column's unit, and from there to its second one
    const int first = kInterleaved || turns ? i * V : a.R + (i - turning) * V;
    const int behind = (a.D - a.R) / V;                     // units behind R, the first half of them paired with the rest
    const int delta = kInterleaved ? 0 : turns ? half : (behind + 1) / 2 * V;
    const bool two = !kInterleaved && (turns || first + delta < a.D);
    const int k_head = a.Hq, v_head = a.Hq + a.Hkv, heads = a.Hq + 2 * a.Hkv;
    const int step = per * (int)gridDim.y, row = a.B * a.D;
    for (int t = 0; t < nt; ++t) {
        const int64_t slot = slots[t];
        if (slot < 0) continue;
        const int64_t blk = slot / a.B;
        const size_t place = ((size_t)blk * a.Hkv * a.B + (size_t)(slot - blk * a.B)) * a.D + first;  // head 0's row
        // each kind's head 0 stands at its own number, so that head h is `h * D` (or rows of the cache) on
        const T *q = static_cast<const T *>(a.q) + (size_t)(t0 + t) * a.q_stride + first;
        const T *k = static_cast<const T *>(a.k) + (size_t)(t0 + t) * a.k_stride + first - (ptrdiff_t)k_head * a.D;
        const T *v = static_cast<const T *>(a.v) + (size_t)(t0 + t) * a.v_stride + first - (ptrdiff_t)v_head * a.D;
        T *qo = static_cast<T *>(a.q_out) + (size_t)(t0 + t) * a.q_out_stride + first;
        T *kc = static_cast<T *>(a.k_cache) + place - (ptrdiff_t)k_head * row;
        T *vc = static_cast<T *>(a.v_cache) + place - (ptrdiff_t)v_head * row;
        const float2 *w = cs + t * half + i * kAngles;
        for (int h = blockIdx.y * per + h0; h < heads; h += kU * step) {
            uint4 x[kU], y[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int n = h + u * step;
                if (n < heads) {
                    const T *from = (n < k_head ? q : n < v_head ? k : v) + (ptrdiff_t)n * a.D;
                    x[u] = *reinterpret_cast<const uint4 *>(from);
                    if (two) y[u] = *reinterpret_cast<const uint4 *>(from + delta);
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int n = h + u * step;
                if (n < heads) {
                    if (turns && n < v_head) {
                        float f[V], g[V];
                        Elem<T>::unpack(x[u], f);
                        if (!kInterleaved) Elem<T>::unpack(y[u], g);
#pragma unroll
                        for (int e = 0; e < kAngles; ++e) {
                            float &p = kInterleaved ? f[2 * e] : f[e], &r = kInterleaved ? f[2 * e + 1] : g[e];
                            if (kInterleaved && e >= live) continue;
                            const float2 t = turned(p, r, w[e]);
                            p = t.x, r = t.y;
                        }
                        const uint4 packed = Unit<T>::pack(f);
                        if constexpr (kInterleaved) {  // the words of pairs behind R stay as they are
                            constexpr int kWords = 4 / kAngles;  // of a pair
                            x[u].x = packed.x;
                            if (1 / kWords < live) x[u].y = packed.y;
                            if (2 / kWords < live) x[u].z = packed.z;
                            if (3 / kWords < live) x[u].w = packed.w;
                        } else {
                            x[u] = packed;
                        }
                        if (!kInterleaved) y[u] = Unit<T>::pack(g);
                    }
                    T *to = n < k_head ? qo + (ptrdiff_t)n * a.D : (n < v_head ? kc : vc) + (ptrdiff_t)n * row;
                    *reinterpret_cast<uint4 *>(to) = x[u];
                    if (two) *reinterpret_cast<uint4 *>(to + delta) = y[u];
                }
            }
        }
    }
}

// Whole heads of 16-bit elements in halves: every column is two units that turn together (upq of them a head).  The tokens' heads stand in one line,
// m = t * heads + head; a thread takes every step-th of them, kU a round.  The first round's loads need no slot and no
// angle, so they are under way before those are there; (cos, sin) lie so that lanes next to each other read neighbours.
// (8192 tokens of 32 + 8 heads, bf16: 36.6 us, 50.3 in rope_units_kernel; of 32 + 32 heads of 64, f16, 32.5 and 41.5.
// Elsewhere this form loses: 32 + 32 heads, 64 of 128 elements turned, 69.6 and 63.2, as neighbouring pairs 85.5 and 63.6;
// 4096 tokens of 32 + 32 whole fp32 heads 70.0 and 65.4.)
template <typename T>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_whole_kernel(const RopeArgs a, int tokens, int upq) {
    constexpr int V = Unit<T>::kN, kU = 4;
    extern __shared__ float2 cs[];  // [tokens][V][upq]
    __shared__ int64_t places[kTokens];  // of each token's row of KV head 0, or -1 for padding
    const int half = a.R / 2, tid = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
    const int i = tid % upq, per = kRopeThreads / upq, h0 = tid / upq, first = i * V;
    const int k_head = a.Hq, v_head = a.Hq + a.Hkv, heads = a.Hq + 2 * a.Hkv;
    const int step = per * (int)gridDim.y, row = a.B * a.D, all = nt * heads;
    uint4 x[kU], y[kU];
    auto load = [&](int m0) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int m = m0 + u * step;
            if (m < all) {
                const int t = m >= heads ? 1 : 0, n = m - t * heads;
                const T *from = n < k_head   ? static_cast<const T *>(a.q) + (size_t)(t0 + t) * a.q_stride + (ptrdiff_t)n * a.D
                                : n < v_head ? static_cast<const T *>(a.k) + (size_t)(t0 + t) * a.k_stride + (ptrdiff_t)(n - k_head) * a.D
                                             : static_cast<const T *>(a.v) + (size_t)(t0 + t) * a.v_stride + (ptrdiff_t)(n - v_head) * a.D;
                x[u] = *reinterpret_cast<const uint4 *>(from + first);
                y[u] = *reinterpret_cast<const uint4 *>(from + first + half);
            }
        }
    };
    const int m0 = blockIdx.y * per + h0;
    if (h0 < per) load(m0);
    if (tid < nt) {
        const int64_t slot = token_slot(a, t0 + tid, blockIdx.y == 0), blk = slot / a.B;
        places[tid] = slot < 0 ? -1 : (blk * a.Hkv * a.B + (slot - blk * a.B)) * a.D;
    }
    for (int e = tid; e < nt * half; e += kRopeThreads) {
        const int t = e / half, p = e - t * half;
        cs[(t * V + p % V) * upq + p / V] = turn_at(turn_fraction(a.freqs[p]), pair_position(a, t0 + t, p), a.mscale);
    }
    __syncthreads();
    if (h0 >= per) return;
    for (int m1 = m0; m1 < all; m1 += kU * step) {
        if (m1 != m0) load(m1);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int m = m1 + u * step;
            if (m >= all) break;
            const int t = m >= heads ? 1 : 0, n = m - t * heads;
            const int64_t place = places[t];
            if (place < 0) continue;
            if (n < v_head) {
                const float2 *w = cs + t * V * upq + i;
                float f[V], g[V];
                Elem<T>::unpack(x[u], f);
                Elem<T>::unpack(y[u], g);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 c = w[e * upq];
                    const float2 r = turned(f[e], g[e], c);
                    f[e] = r.x, g[e] = r.y;
                }
                x[u] = Unit<T>::pack(f);
                y[u] = Unit<T>::pack(g);
            }
            T *to = n < k_head ? static_cast<T *>(a.q_out) + (size_t)(t0 + t) * a.q_out_stride + (ptrdiff_t)n * a.D
                               : static_cast<T *>(n < v_head ? a.k_cache : a.v_cache) + place + (ptrdiff_t)(n < v_head ? n - k_head : n - v_head) * row;
            *reinterpret_cast<uint4 *>(to + first) = x[u];
            *reinterpret_cast<uint4 *>(to + first + half) = y[u];
        }
    }
}

// Halves that are not whole units: a thread takes one unit of a head and its elements' partners
// R / 2 away one by one.  grid: (tokens, parts of their heads); a CTA takes `per` whole heads at
// a time, and stores them once all of it has read them (q_out may be q).
// Measured: 8192 tokens of 32 + 32 heads (D 128, f16, 20 elements rotated) 106 us, of 32 + 8 heads, 74 elements, 69;
// two or three rounds of heads in flight 112 and 111; element by element 228.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_split_kernel(const RopeArgs a, int upq) {
    constexpr int V = Unit<T>::kN;
    __shared__ float2 cs[kMaxPairs];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x, tid = threadIdx.x, half = a.R / 2;
    const int64_t slot = token_slot(a, t, tid == 0 && blockIdx.y == 0);
    if (slot < 0) return;
    for (int p = tid; p < half; p += kRopeThreads)
        cs[p] = turn_at(turn_fraction(a.freqs[p]), pair_position(a, t, p), a.mscale);
    __syncthreads();
    const int64_t blk = slot / a.B, off = slot % a.B;
    const int i = tid % upq, per = kRopeThreads / upq, h0 = tid / upq, d0 = i * V;
    const int k_head = a.Hq, v_head = a.Hq + a.Hkv, heads = a.Hq + 2 * a.Hkv;
    for (int g = blockIdx.y * per; g < heads; g += (int)gridDim.y * per) {
        const int n = g + h0;
        const bool mine = h0 < per && n < heads;
        const int at = n < k_head ? n : n < v_head ? n - k_head : n - v_head;  // within q, k or v
        union {
            uint4 raw;
            T e[V];
        } x;
        if (mine) {
            const T *head = (n < k_head   ? static_cast<const T *>(a.q) + (size_t)t * a.q_stride
                             : n < v_head ? static_cast<const T *>(a.k) + (size_t)t * a.k_stride
                                          : static_cast<const T *>(a.v) + (size_t)t * a.v_stride) +
                            (size_t)at * a.D;
            x.raw = *reinterpret_cast<const uint4 *>(head + d0);
            if (n < v_head) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int d = d0 + e;
                    if (d >= a.R) break;
                    const bool low = d < half;
                    const float2 c = cs[low ? d : d - half];
                    const float other = static_cast<float>(head[low ? d + half : d - half]), own = static_cast<float>(x.e[e]);
                    x.e[e] = narrow<T>(low ? turned(own, other, c).x : turned(other, own, c).y);
                }
            }
        }
        __syncthreads();
        if (mine) {
            T *to = n < k_head ? static_cast<T *>(a.q_out) + (size_t)t * a.q_out_stride + (size_t)at * a.D
                               : static_cast<T *>(n < v_head ? a.k_cache : a.v_cache) +
                                     (((size_t)blk * a.Hkv + at) * a.B + off) * a.D;
            *reinterpret_cast<uint4 *>(to + d0) = x.raw;
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

// The unit kernels want the whole L1 for their loads in flight, also right after a kernel
// that asked for a large part of it as shared memory.
template <typename T, void (*kKernel)(RopeArgs, int, int)>
cudaError_t launch_units(const RopeArgs &a, int tokens, int upq, dim3 grid, size_t smem, cudaStream_t st) {
    static std::atomic<int> configured[kMaxLaunchDevices];
    int one = 0;
    const cudaError_t e = per_device_value(configured, &one, [](int, int *v) {
        *v = 1;
        return cudaFuncSetAttribute(kKernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxL1);
    });
    if (e != cudaSuccess) return e;
    return launch_rope(kKernel, grid, smem, st, a, tokens, upq);
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs &a, cudaStream_t st) {
    constexpr int V = Unit<T>::kN;
    const bool whole = a.interleaved || a.R % (2 * V) == 0;
    const int upq = a.interleaved || !whole ? a.D / V : a.R / 2 / V + ((a.D - a.R) / V + 1) / 2;
    if (upq > kRopeThreads) return launch_rope(rope_elements_kernel<T>, dim3((unsigned)a.T), 0, st, a);
    if (!whole) {
        // few tokens: their heads over several CTAs
        const int per = kRopeThreads / upq, passes = (a.Hq + 2 * a.Hkv + per - 1) / per;
        const int parts = 4 * 152 / a.T;
        return launch_rope(rope_split_kernel<T>, dim3((unsigned)a.T, (unsigned)(parts < 1 ? 1 : parts < passes ? parts : passes)),
                           0, st, a, upq);
    }
    // Few tokens: their heads over several CTAs, down to one head a thread, so that a step's loads are
    // all in flight at once.  Many: two tokens a CTA, whose slots, positions and angles then cost one
    // chain of loads and one barrier (8192 tokens: 64 us; one token a CTA 72, three 65, four 70, eight 85).
    const int tokens = a.T >= 16 * 152 && a.R <= 1024 ? kTokens : 1;
    const int groups = (a.T + tokens - 1) / tokens, per = kRopeThreads / upq;
    const int passes = (a.Hq + 2 * a.Hkv + per - 1) / per;
    int parts = (4 * 152 + groups - 1) / groups;
    parts = parts < passes ? parts : passes;
    const dim3 grid((unsigned)groups, (unsigned)(parts > 0 ? parts : 1));
    const size_t smem = (size_t)tokens * (a.R / 2) * sizeof(float2);
    if (a.interleaved) return launch_units<T, rope_units_kernel<T, true>>(a, tokens, upq, grid, smem, st);
    if constexpr (sizeof(T) == 2)
        if (a.R == a.D) return launch_units<T, rope_whole_kernel<T>>(a, tokens, upq, grid, smem, st);
    return launch_units<T, rope_units_kernel<T, false>>(a, tokens, upq, grid, smem, st);
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
