// pa_scored_finish.cu -- the last launch of scored attention.
//
// Merge: for a row whose keys lie in several partitions,
//   o = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p,   M = max_p m_p,
// over the partitions p0 .. p1 that the row's range touches (m in log2 units;
// a partition that saw no key has m = -inf and weight 0).
// Sums: with M and L = sum_p 2^(m_p - M) l_p of each of the G query heads of a KV
// head, every key j that the decode row saw gets
//   sums[row, kvh, j] += sum_g 2^(z_gj - M_g) / L_g
// from the logits z that the partition kernel left (4 bytes per query head and
// key, against 2 D elements of K and V that a second pass would read again).
#include "pa_score.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 4 * kThreads;  // keys of one block of the sums

// Maximum and sum over partitions p0 .. p1 of the (m, l) pairs at ml.  Whole warp.
__device__ __forceinline__ float2 merged_ml(const float *ml, int p0, int p1, int lane) {
    float M = -INFINITY, L = 0.f;
    for (int p = p0 + lane; p <= p1; p += 32) M = fmaxf(M, ml[2 * p]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;  // nothing seen, or NaN logits alone: weights 0, and l as it is
    for (int p = p0 + lane; p <= p1; p += 32) L += ex2(ml[2 * p] - M) * ml[2 * p + 1];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    return make_float2(M, L);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) scored_finish_kernel(const ScoredArgs a, int merge_blocks, int tiles) {
    constexpr int kPer = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = a.max_blocks * a.B;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.query_start && a.plan_hdr[0] < 0) return;
    if ((int)blockIdx.x < merge_blocks) {
        const long long w = (long long)blockIdx.x * (kThreads / 32) + warp;
        if (w >= (long long)a.T * a.Hq) return;
        const int i = (int)(w / a.Hq);
        const RowOf r = row_of(a, i, cap);
        if (r.s < 0) return;
        const int2 range = row_range(a, i, r.pos, r.len);
        if (range.x >= range.y) return;
        const int p0 = range.x / a.partition_size, p1 = (range.y - 1) / a.partition_size;
        if (p0 == p1) return;  // written in place
        const float *ml = a.ws_ml + 2 * w * a.max_parts;
        const float *acc = a.ws_acc + (size_t)w * a.max_parts * D + lane * kPer;
        const float2 t = merged_ml(ml, p0, p1, lane);
        float o[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = 0.f;
        for (int p = p0; p <= p1; ++p) {
            const float wt = ex2(ml[2 * p] - t.x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] = fmaf(wt, acc[(size_t)p * D + e], o[e]);
        }
        const float inv = t.y != 0.f ? 1.f / t.y : 0.f;
        const size_t at = (size_t)w * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            if (a.out16) store_out(static_cast<T *>(a.out) + at + e, o[e] * inv);
            else static_cast<float *>(a.out)[at + e] = o[e] * inv;
        }
        return;
    }
    // ---- sums of one (sequence, KV head), kTile keys
    const int b = (int)blockIdx.x - merge_blocks;
    const int s = b / tiles / a.Hkv, kvh = b / tiles % a.Hkv;
    const int G = a.Hq / a.Hkv;
    const RowOf r = row_of(a, s, cap);
    const int2 range = row_range(a, s, r.pos, r.len);
    const int k0 = (range.x & ~3) + (b % tiles) * kTile;
    if (range.x >= range.y || k0 >= range.y) return;
    const int row = a.sum_rows ? a.sum_rows[s] : s;
    if (row < 0 || row >= a.sum_num_rows) {
        if (threadIdx.x == 0) set_error(a.err, PA_DEVERR_BAD_ROW);
        return;
    }
    __shared__ float2 tot[8];
    if (warp < G) {
        const int p0 = range.x / a.partition_size, p1 = (range.y - 1) / a.partition_size;
        const float2 t = merged_ml(a.ws_ml + 2 * ((size_t)s * a.Hq + kvh * G + warp) * a.max_parts, p0, p1, lane);
        if (lane == 0) tot[warp] = make_float2(t.x, t.y != 0.f ? 1.f / t.y : 0.f);
    }
    __syncthreads();
    const int j = k0 + 4 * threadIdx.x;
    if (j >= range.y) return;
    float *dst = a.sums + ((size_t)row * a.Hkv + kvh) * a.sum_cols + j;
    float add[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < G; ++g) {
        const float4 z = *reinterpret_cast<const float4 *>(a.ws_logits + ((size_t)s * a.Hq + kvh * G + g) * cap + j);
        const float2 t = tot[g];
        add[0] += ex2(z.x - t.x) * t.y;
        add[1] += ex2(z.y - t.x) * t.y;
        add[2] += ex2(z.z - t.x) * t.y;
        add[3] += ex2(z.w - t.x) * t.y;
    }
    // keys outside the range have no logit: what the workspace holds there is not used
    float4 v = *reinterpret_cast<float4 *>(dst);
    if (j >= range.x && j < range.y) v.x += add[0];
    if (j + 1 >= range.x && j + 1 < range.y) v.y += add[1];
    if (j + 2 >= range.x && j + 2 < range.y) v.z += add[2];
    if (j + 3 >= range.x && j + 3 < range.y) v.w += add[3];
    *reinterpret_cast<float4 *>(dst) = v;
}

template <typename T>
cudaError_t launch_finish_t(const ScoredArgs &a, cudaStream_t st) {
    const long long warps = (long long)a.T * a.Hq;
    const int merge = a.max_parts > 1 ? (int)((warps + kThreads / 32 - 1) / (kThreads / 32)) : 0;
    const int cap = a.max_blocks * a.B;
    const int tiles = a.sums ? (cap + 3 + kTile - 1) / kTile : 0;
    const long long blocks = merge + (long long)a.S * a.Hkv * tiles * (a.sums ? 1 : 0);
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.D == 64) return cudaLaunchKernelEx(&cfg, scored_finish_kernel<T, 64>, a, merge, tiles);
    if (a.D == 128) return cudaLaunchKernelEx(&cfg, scored_finish_kernel<T, 128>, a, merge, tiles);
    return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_scored_finish(const ScoredArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_finish_t<__nv_bfloat16>(a, st) : launch_finish_t<__half>(a, st);
}

}  // namespace pa
