// pa_rope.cu -- rotary positions of new queries and keys, and the write of keys
// and values into their cache slots, in one pass.
//
// Pair (a, b) of a head at angle t = pos * freq becomes mscale * (a cos t -
// b sin t, b cos t + a sin t).  The angle is reduced in 64 bits: pos * freq / 2 pi
// minus its nearest whole number is a fraction of a turn known to about 2^-30
// even at pos = 2^20, and sincospif of twice that fraction loses nothing more
// than fp32 has.  One CTA computes a token's R / 2 (cos, sin) pairs into shared
// memory once and uses them for all of its heads.
#include "pa_device.cuh"
#include "pa_scored.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 1024;

template <typename T>
struct Narrow;
template <>
struct Narrow<float> {
    static __device__ __forceinline__ float to(float x) { return x; }
};
template <>
struct Narrow<__half> {
    static __device__ __forceinline__ __half to(float x) { return __float2half_rn(x); }
};
template <>
struct Narrow<__nv_bfloat16> {
    static __device__ __forceinline__ __nv_bfloat16 to(float x) { return __float2bfloat16_rn(x); }
};

// One CTA per token: heads 0 .. Hq-1 are queries, the next Hkv keys, the last
// Hkv values (copied).  An element at a time.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kv_kernel(const RopeArgs a) {
    __shared__ float2 cs[kMaxPairs];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x;
    const int64_t slot = a.slots[t];
    if (slot < 0) return;
    if (slot >= (int64_t)a.N * a.B) {
        if (threadIdx.x == 0) set_error(a.err, PA_DEVERR_BAD_SLOT);
        return;
    }
    const int half = a.R / 2;
    const double pos = (double)a.positions[t];
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        const double turns = pos * a.freqs[i] * 0.15915494309189535;  // 1 / (2 pi)
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[i] = make_float2(c * a.mscale, s * a.mscale);
    }
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
            dst[ia] = Narrow<T>::to(x * w.x - y * w.y);
            dst[ib] = Narrow<T>::to(y * w.x + x * w.y);
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
cudaError_t launch_rope_t(const RopeArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_write_kv_kernel<T>, a);
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
