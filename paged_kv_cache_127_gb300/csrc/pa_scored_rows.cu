// pa_scored_rows.cu -- scored attention on the CUDA cores, one CTA per (query
// row, KV head, context partition).
//
// For row i at position pos, the G query heads of a KV head and the keys j of
// one partition inside the row's range:
//   z = scale q.k_j, capped by softcap tanh(z / softcap), minus slope |pos - j|
//   m = max z, l = sum exp(z - m), acc = sum exp(z - m) v_j
// all in fp32, with logits kept in log2 units so that an exponential is one ex2.
// Warp w takes query heads w, w + 4 and walks the partition in tiles of 32
// keys: lane j computes key j's logit (its K row as 16-byte loads), the
// tile's maximum and sum are warp reductions, and for P V a lane owns D / 32
// columns while the weights come by shuffle.  Keys outside the range are never
// loaded, so what they hold does not matter.  A row whose range lies in one
// partition is written at once; else (m, l, acc) go to the merge
// (pa_scored_finish.cu).
#include "pa_score.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;

// A lane's N neighbouring elements of a V row, in one load.
template <typename T, int N>
struct Row {
    float f[N];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = 0.f;
    }
    __device__ __forceinline__ void load(const T *p) {
        struct alignas(sizeof(T) * N) Vec {
            T e[N];
        };
        const Vec v = *reinterpret_cast<const Vec *>(p);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = static_cast<float>(v.e[e]);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) scored_rows_kernel(const ScoredArgs a) {
    constexpr int kVec = Elem<T>::kVec;
    constexpr int kPer = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv, part = blockIdx.y;
    const int G = a.Hq / a.Hkv, B = a.B, cap = a.max_blocks * a.B;
    if (!a.query_start && part == 0 && kvh == 0 && threadIdx.x == 0) {
        const int len = a.context_lens[i];
        if (len < 0 || len > cap) set_error(a.err, PA_DEVERR_BAD_LEN);
    }
    if (a.query_start && a.plan_hdr[0] < 0) return;  // query_start refused by the check kernel
    const RowOf r = row_of(a, i, cap);
    if (r.s < 0) return;
    const int2 range = row_range(a, i, r.pos, r.len);
    if (range.x >= range.y) {
        if (part == 0)
            for (int d = threadIdx.x; d < G * D; d += blockDim.x) {
                const size_t o = ((size_t)i * a.Hq + kvh * G) * D + d;
                if (a.out16) store_out(static_cast<T *>(a.out) + o, 0.f);
                else static_cast<float *>(a.out)[o] = 0.f;
            }
        return;
    }
    const int Pt = a.partition_size;
    const int p0 = range.x / Pt, p1 = (range.y - 1) / Pt;
    if (part < p0 || part > p1) return;
    const int k0 = max(range.x, part * Pt), k1 = min(range.y, (part + 1) * Pt);
    const int32_t *row = a.block_tables + (size_t)r.s * a.max_blocks;
    const T *kc = static_cast<const T *>(a.k_cache);
    const T *vc = static_cast<const T *>(a.v_cache);

    for (int g = warp; g < G; g += kWarps) {
        const int h = kvh * G + g;
        const T *q = static_cast<const T *>(a.q) + ((size_t)i * a.Hq + h) * D;
        const float slope = a.slopes ? a.slopes[h] * kLog2e : 0.f;
        float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
        for (int t0 = k0; t0 < k1; t0 += 32) {
            const int j = t0 + lane;
            float z = -INFINITY;
            size_t off = 0;
            bool in = j < k1;
            if (in) {
                const int blk = row[j / B];
                if (blk < 0 || blk >= a.N) {
                    set_error(a.err, PA_DEVERR_BAD_BLOCK);
                    in = false;
                } else {
                    off = (((size_t)blk * a.Hkv + kvh) * B + j % B) * D;
                }
            }
            if (in) {
                float dot = 0.f;
#pragma unroll 8
                for (int c = 0; c < D / kVec; ++c) {
                    float qf[kVec], kf[kVec];
                    Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(q) + c), qf);
                    Elem<T>::unpack(*(reinterpret_cast<const uint4 *>(kc + off) + c), kf);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) dot = fmaf(qf[e], kf[e], dot);
                }
                z = dot * a.scale;
                if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
                z = z * kLog2e - slope * fabsf((float)(r.pos - j));
            }
            if (a.ws_logits && j < k1) a.ws_logits[((size_t)r.s * a.Hq + h) * cap + j] = z;
            float mx = z;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m, mx);
            const float mu = mn == -INFINITY ? 0.f : mn;
            const float al = ex2(m - mu);  // 0 while m is -inf
            const float p = ex2(z - mu);
            float ps = p;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
            l = l * al + ps;
            m = mn;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] *= al;
            const unsigned have = __ballot_sync(0xffffffffu, in);
            // eight rows of V in flight; keys without a row (weight 0) load none
            const int last = 32 - __clz(have);
            for (int t0v = 0; t0v < last; t0v += 8) {
                Row<T, kPer> v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const size_t vo = __shfl_sync(0xffffffffu, (unsigned long long)off, t0v + u);
                    if (have >> (t0v + u) & 1) v[u].load(vc + vo + lane * kPer);
                    else v[u].zero();
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float pt = __shfl_sync(0xffffffffu, p, t0v + u);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) acc[e] = fmaf(pt, v[u].f[e], acc[e]);
                }
            }
        }
        const size_t o = ((size_t)i * a.Hq + h) * D + lane * kPer;
        const size_t w = ((size_t)i * a.Hq + h) * a.max_parts + part;
        if (p0 == p1) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const float x = l != 0.f ? acc[e] / l : 0.f;
                if (a.out16) store_out(static_cast<T *>(a.out) + o + e, x);
                else static_cast<float *>(a.out)[o + e] = x;
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) a.ws_acc[w * D + lane * kPer + e] = acc[e];
        }
        if ((p0 != p1 || a.ws_logits) && lane == 0) *reinterpret_cast<float2 *>(a.ws_ml + 2 * w) = make_float2(m, l);
    }
}

// Chunk calls without a plan: flag bad ranges and lengths once; plan_hdr[0] < 0
// when query_start is not non-decreasing within [0, T].
__global__ void __launch_bounds__(1024) scored_check_kernel(const ScoredArgs a) {
    const int cap = a.max_blocks * a.B;
    int bad = threadIdx.x == 0 && (a.query_start[0] < 0 || a.query_start[a.S] > a.T);
    for (int s = threadIdx.x; s < a.S; s += blockDim.x) bad |= a.query_start[s] > a.query_start[s + 1];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.plan_hdr[0] = bad ? -1 : 0;
        if (bad) set_error(a.err, PA_DEVERR_BAD_LEN);
    }
    if (bad) return;
    for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
        const int len = a.context_lens[s], n = a.query_start[s + 1] - a.query_start[s];
        if (len < 0 || len > cap || n > len || n > a.max_query_len) set_error(a.err, PA_DEVERR_BAD_LEN);
    }
}

template <typename T>
cudaError_t launch_rows_t(const ScoredArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)((long long)a.T * a.Hkv), (unsigned)a.max_parts);
    if (a.D == 64) scored_rows_kernel<T, 64><<<grid, kWarps * 32, 0, st>>>(a);
    else if (a.D == 128) scored_rows_kernel<T, 128><<<grid, kWarps * 32, 0, st>>>(a);
    else return cudaErrorNotSupported;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scored_rows(const ScoredArgs &a, int dtype, cudaStream_t st) {
    if (a.query_start) {
        scored_check_kernel<<<1, 1024, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (dtype == PA_F32) return launch_rows_t<float>(a, st);
    if (dtype == PA_F16) return launch_rows_t<__half>(a, st);
    return launch_rows_t<__nv_bfloat16>(a, st);
}

}  // namespace pa
