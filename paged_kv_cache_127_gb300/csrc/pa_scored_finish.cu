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
//
// Bound: latency of short chains of loads.  Measured alone, caches cold: the sums of 256 sequences of 800
// tokens on average 20 us, of 32 windows of 4096 keys 18 us; the merges of such batches 6 to 9 us.
#include "pa_mma.cuh"
#include "pa_score.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;

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

// The running sums of four keys and the logits of the G heads for them.
template <int G>
struct KeySpan {
    float4 v, x[G];
    __device__ __forceinline__ void load(const float *sums, const float *z, size_t heads, int j) {
        v = *reinterpret_cast<const float4 *>(sums + j);
#pragma unroll
        for (int g = 0; g < G; ++g) x[g] = *reinterpret_cast<const float4 *>(z + g * heads + j);
    }
    // += sum over the heads of 2^(z - M) / L for the keys of [begin, end); keys
    // outside have no logit (whatever the workspace holds there is not used)
    __device__ __forceinline__ void add(float *sums, const float2 *tot, int j, int begin, int end) {
        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float2 t = tot[g];
            w[0] += ex2(x[g].x - t.x) * t.y;
            w[1] += ex2(x[g].y - t.x) * t.y;
            w[2] += ex2(x[g].z - t.x) * t.y;
            w[3] += ex2(x[g].w - t.x) * t.y;
        }
        if (j >= begin) v.x += w[0];
        if (j + 1 >= begin && j + 1 < end) v.y += w[1];
        if (j + 2 >= begin && j + 2 < end) v.z += w[2];
        if (j + 3 >= begin && j + 3 < end) v.w += w[3];
        *reinterpret_cast<float4 *>(sums + j) = v;
    }
};

// One block per (query row, KV head) and, with sums, part of the row's keys: the
// G heads' (M, L) once for the merge and the sums.  The first four keys of a
// thread are loaded before the totals are known, so that a block pays one chain of loads
// where its part is short.  (Loading each next four while the last are added cost registers:
// 108 us a call against 107 on 32 windows of 4096 keys.)
template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads) scored_finish_kernel(const ScoredArgs a, int splits, int merges) {
    __shared__ float2 tot[G];  // (M, 1 / L) of each head of the group
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % splits, kvh = blockIdx.x / splits % a.Hkv, i = blockIdx.x / splits / a.Hkv;
    const int cap = a.max_blocks * a.B, P = a.max_parts;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.query_start && a.plan_hdr[0] < 0) return;
    const RowOf r = row_of(a, i, cap);
    if (r.s < 0) return;
    const int2 range = row_range(a, i, r.pos, r.len);
    if (range.x >= range.y) return;
    int p0 = range.x / a.partition_size, p1 = (range.y - 1) / a.partition_size;
    if (a.listed) {
        p0 = 0;
        p1 = pieces_of(range, a.partition_size, a.plan_hdr[3]) - 1;
    }
    const bool merge = merges && p0 != p1 && split == 0;  // else written in place, by another block or the merge kernel
    if (!merge && !a.sums) return;
    const size_t head0 = (size_t)i * a.Hq + kvh * G;
    const int row = a.sums ? (a.sum_rows ? a.sum_rows[i] : i) : -1;
    const bool add = row >= 0 && row < a.sum_num_rows;
    if (a.sums && !add && threadIdx.x == 0) set_error(a.err, PA_DEVERR_BAD_ROW);
    float *sums = a.sums + ((size_t)(add ? row : 0) * a.Hkv + kvh) * a.sum_cols;
    const float *z = a.ws_logits + head0 * cap;
    int j = (range.x & ~3) + 4 * (split * kThreads + (int)threadIdx.x);
    KeySpan<G> cur;
    if (add && j < range.y) cur.load(sums, z, cap, j);
    if (warp < G) {
        const float2 t = merged_ml(a.ws_ml + 2 * (head0 + warp) * P, p0, p1, lane);
        if (lane == 0) tot[warp] = make_float2(t.x, t.y != 0.f ? 1.f / t.y : 0.f);
    }
    __syncthreads();
    if (merge) {
        for (int c = threadIdx.x; c < G * D / 4; c += kThreads) {
            const int g = c / (D / 4), d = c % (D / 4) * 4;
            const float *ml = a.ws_ml + 2 * (head0 + g) * P;
            const float *acc = a.ws_acc + (head0 + g) * P * D + d;
            const float2 t = tot[g];
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int p = p0; p <= p1; ++p) {
                const float w = ex2(ml[2 * p] - t.x);
                const float4 x = *reinterpret_cast<const float4 *>(acc + (size_t)p * D);
                o.x = fmaf(w, x.x, o.x);
                o.y = fmaf(w, x.y, o.y);
                o.z = fmaf(w, x.z, o.z);
                o.w = fmaf(w, x.w, o.w);
            }
            const size_t at = (head0 + g) * D + d;
            if (a.out16) {
                const uint2 y = make_uint2(Mma16<T>::pack(o.x * t.y, o.y * t.y), Mma16<T>::pack(o.z * t.y, o.w * t.y));
                *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + at) = y;
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) =
                    make_float4(o.x * t.y, o.y * t.y, o.z * t.y, o.w * t.y);
            }
        }
    }
    if (!add) return;
    const int step = 4 * kThreads * splits;
    while (j < range.y) {
        cur.add(sums, tot, j, range.x, range.y);
        j += step;
        if (j < range.y) cur.load(sums, z, cap, j);
    }
}

template <typename T, int D>
cudaError_t launch_finish_t(const ScoredArgs &a, bool merges, cudaStream_t st) {
    if (a.max_parts == 1 && !a.sums) return cudaSuccess;
    const long long pairs = (long long)a.T * a.Hkv;
    // Blocks for the sums: up to 8 per SM (4 are resident), so that a few long sequences fill the GPU,
    // at most one per 1024 positions of the tables.  One block per 1024 positions whatever
    // the batch took 35 us on 256 sequences of up to 4096 tokens (8,192 blocks, most
    // with no keys, each paying the chain of loads up to the heads' totals).
    long long splits = 1;
    if (a.sums) {
        const long long most = ((long long)a.max_blocks * a.B + 4 * kThreads - 1) / (4 * kThreads);
        splits = 8 * 152 / pairs;
        splits = splits < 1 ? 1 : (splits > most ? most : splits);
    }
    if (pairs * splits > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * splits));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (a.Hq / a.Hkv) {
        case 1: return cudaLaunchKernelEx(&cfg, scored_finish_kernel<T, D, 1>, a, (int)splits, (int)merges);
        case 2: return cudaLaunchKernelEx(&cfg, scored_finish_kernel<T, D, 2>, a, (int)splits, (int)merges);
        case 4: return cudaLaunchKernelEx(&cfg, scored_finish_kernel<T, D, 4>, a, (int)splits, (int)merges);
        case 8: return cudaLaunchKernelEx(&cfg, scored_finish_kernel<T, D, 8>, a, (int)splits, (int)merges);
        default: return cudaErrorNotSupported;
    }
}

// Partials p0 .. p0 + N - 1 (those below np) of one (row, head): every load first,
// then the sums in partition order.
template <int D, int N>
__device__ __forceinline__ void merge_short(const float *ml, const float *acc, int np, float (&o)[D / 32], float &L) {
    constexpr int kPer = D / 32;
    float2 w[N];
    float x[N][kPer];
#pragma unroll
    for (int p = 0; p < N; ++p)
        if (p < np) {
            w[p] = *reinterpret_cast<const float2 *>(ml + 2 * p);
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(acc + (size_t)p * D + e);
                x[p][e] = v.x;
                x[p][e + 1] = v.y;
            }
        }
    float M = -INFINITY;
#pragma unroll
    for (int p = 0; p < N; ++p)
        if (p < np) M = fmaxf(M, w[p].x);
    if (M == -INFINITY) M = 0.f;
#pragma unroll
    for (int p = 0; p < N; ++p)
        if (p < np) {
            const float t = ex2(w[p].x - M);
            L = fmaf(t, w[p].y, L);
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] = fmaf(t, x[p][e], o[e]);
        }
}

// Partials p0, p0 + step, ... below np of one (row, head), against the maximum M known beforehand.
template <int D>
__device__ __forceinline__ void merge_long(const float *ml, const float *acc, int p0, int step, int np, float M,
                                           float (&o)[D / 32]) {
    constexpr int kPer = D / 32;
    constexpr int kU = 8;
    for (int p = p0; p < np; p += kU * step) {
        float w[kU], x[kU][kPer];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int q = p + u * step;
            w[u] = -INFINITY;
            if (q < np) {
                w[u] = ml[2 * q];
#pragma unroll
                for (int e = 0; e < kPer; e += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(acc + (size_t)q * D + e);
                    x[u][e] = v.x;
                    x[u][e + 1] = v.y;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (p + u * step < np) {
                const float t = ex2(w[u] - M);
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] = fmaf(t, x[u][e], o[e]);
            }
    }
}

// Listed (row, head) pairs, lane i owning D / 32 columns; the blocks stride over the list.  One
// warp each, or, while the pairs are fewer than the blocks, a whole block each, whose warps
// share the partitions: a few long sequences have hundreds, and one warp's chain of loads over them took
// longer than the attention (4 sequences of 20,000 tokens on average: 109 us a call).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) scored_merge_kernel(const ScoredArgs a) {
    constexpr int kPer = D / 32, kWarps = kThreads / 32;
    __shared__ float part[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long n = (long long)a.plan_hdr[2] * a.Hq;
    const bool shared = n <= gridDim.x;
    const long long step = shared ? gridDim.x : (long long)gridDim.x * kWarps;
    for (long long w = shared ? blockIdx.x : (long long)blockIdx.x * kWarps + warp; w < n; w += step) {
        const int4 e = a.merge_list[w / a.Hq];
        const size_t head = (size_t)e.x * a.Hq + (int)(w % a.Hq);
        const int np = e.z - e.y + 1;
        const float *ml = a.ws_ml + 2 * (head * a.max_parts + e.y);
        const float *acc = a.ws_acc + (head * a.max_parts + e.y) * D + lane * kPer;
        float o[kPer], L = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = 0.f;
        if (np <= 2) {
            if (!shared || warp == 0) merge_short<D, 2>(ml, acc, np, o, L);
        } else if (np <= 8) {
            if (!shared || warp == 0) merge_short<D, 8>(ml, acc, np, o, L);
        } else {
            const float2 t = merged_ml(ml, 0, np - 1, lane);
            L = t.y;
            merge_long<D>(ml, acc, shared ? warp : 0, shared ? kWarps : 1, np, t.x, o);
            if (shared) {
                __syncthreads();  // the last pair's parts have been read
#pragma unroll
                for (int i = 0; i < kPer; ++i) part[warp][lane * kPer + i] = o[i];
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    o[i] = 0.f;
#pragma unroll
                    for (int v = 0; v < kWarps; ++v) o[i] += part[v][lane * kPer + i];
                }
            }
        }
        if (shared && warp != 0) continue;
        const float inv = L != 0.f ? 1.f / L : 0.f;
        const size_t at = head * D + lane * kPer;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            if (a.out16) *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + at + i) = Mma16<T>::pack(o[i] * inv, o[i + 1] * inv);
            else *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at + i) = make_float2(o[i] * inv, o[i + 1] * inv);
        }
    }
}

template <typename T, int D>
cudaError_t launch_merge_t(const ScoredArgs &a, cudaStream_t st) {
    if (a.max_parts == 1) return cudaSuccess;
    const long long pairs = (long long)a.T * a.Hq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs < 8 * 152 ? pairs : 8 * 152));  // one resident wave at most
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_merge_kernel<T, D>, a);
}

}  // namespace

cudaError_t launch_scored_merge(const ScoredArgs &a, bool bf16, cudaStream_t st) {
    if (a.D == 64) return bf16 ? launch_merge_t<__nv_bfloat16, 64>(a, st) : launch_merge_t<__half, 64>(a, st);
    if (a.D == 128) return bf16 ? launch_merge_t<__nv_bfloat16, 128>(a, st) : launch_merge_t<__half, 128>(a, st);
    return cudaErrorNotSupported;
}

cudaError_t launch_scored_finish(const ScoredArgs &a, bool listed, bool bf16, cudaStream_t st) {
    // Rows of many partitions are merged by the merge kernel, a block each, before the sums; with up to
    // 16 partitions the sums' blocks merge them on the way (one launch less).
    const bool apart = listed && a.max_parts > 16;
    if (apart) {
        const cudaError_t e = launch_scored_merge(a, bf16, st);
        if (e != cudaSuccess) return e;
    }
    if (a.D == 64) return bf16 ? launch_finish_t<__nv_bfloat16, 64>(a, !apart, st) : launch_finish_t<__half, 64>(a, !apart, st);
    if (a.D == 128) return bf16 ? launch_finish_t<__nv_bfloat16, 128>(a, !apart, st) : launch_finish_t<__half, 128>(a, !apart, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
