// pa_scored_rows.cu -- scored attention over fp32 caches on the CUDA cores, one
// CTA per (query row, KV head, context partition).
//
// For row i at position pos, the G query heads of a KV head and the keys j of
// one partition inside the row's range:
//   z = scale q.k_j, capped by softcap tanh(z / softcap), minus slope |pos - j|
//   m = max z, l = sum exp(z - m), acc = sum exp(z - m) v_j
// all in fp32, with logits kept in log2 units so that an exponential is one ex2.
// The partition's tiles of 32 keys go round the warps, all G heads at once, so that each
// K and V row is read once: eight lanes share a K row (whole 128-byte lines), their eight
// partial dots a head are summed and handed out by a transposing butterfly (7 shuffles), after
// which a lane owns one key; the weights pass through shared memory to P V, where a
// lane owns D / 32 columns.  The warps' (m, l, acc) are joined at the end.  Keys outside the
// range are never loaded, so what they hold does not matter.  A row whose range
// lies in one partition is written at once; else (m, l, acc) go to the merge
// (pa_scored_finish.cu).
//
// Bound: for a batch of decodes instruction issue (2 D fused multiply-adds a key and head) beside HBM,
// latency for short sequences; chunk rows each read their keys again (from L2).
// Measured (32 query heads, D 128): 256 sequences, 8 KV heads, 408 us (floor 248; the f32 kernel of
// pa_decode, plain scores, takes 405), 32 KV heads with documents and a bias 264 us (floor 227), a window of
// 4096 with 64 query heads and sums 440 us (floor 160), five drafted tokens of 256 sequences 1270 us; three sequences of
// 12 to 47 tokens 5 us. A warp per query head, re-reading K and V for each, took 1081, 377, 1350, 4562 and 8 us.
#include "pa_score.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;

// N neighbouring floats of a row.
template <int N>
struct alignas(4 * N) Floats {
    float f[N];
};

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// CTAs per SM that the registers are to leave room for, with G heads' partial dots and sums in
// them (256 sequences, G 4: 4 take 406 us, 3 take 515, 5 take 457; G 8, windows: 2 take 440, 4 take 577;
// G 1: 5 take 266, 4 take 282, 6 take 270).
constexpr int row_ctas(int G) { return G == 8 ? 2 : G == 4 ? 4 : 5; }

template <int D, int G>
__global__ void __launch_bounds__(kWarps * 32, row_ctas(G)) scored_rows_kernel(const ScoredArgs a) {
    constexpr int kPer = D / 32;     // columns of a lane in P V
    constexpr int kChunks = D / 32;  // 16-byte chunks of a K row per lane, eight lanes a row
    __shared__ float4 qs[G][D / 4];
    __shared__ float ps[kWarps][G][32];
    __shared__ float2 ml[kWarps][G];
    __shared__ Floats<kPer> accs[kWarps][G][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = blockIdx.x / a.Hkv, kvh = blockIdx.x % a.Hkv, part = blockIdx.y;
    const int B = a.B, cap = a.max_blocks * a.B;
    if (!a.query_start && part == 0 && kvh == 0 && threadIdx.x == 0) {
        const int len = a.context_lens[i];
        if (len < 0 || len > cap) set_error(a.err, PA_DEVERR_BAD_LEN);
    }
    if (a.query_start && a.plan_hdr[0] < 0) return;  // query_start refused by the check kernel
    const RowOf r = row_of(a, i, cap);
    if (r.s < 0) return;
    const int2 range = row_range(a, i, r.pos, r.len);
    float *out = static_cast<float *>(a.out) + ((size_t)i * a.Hq + kvh * G) * D;
    if (range.x >= range.y) {
        if (part == 0)
            for (int d = threadIdx.x; d < G * D; d += blockDim.x) out[d] = 0.f;
        return;
    }
    const int Pt = a.partition_size;
    const int p0 = range.x / Pt, p1 = (range.y - 1) / Pt;
    if (part < p0 || part > p1) return;
    const int k0 = max(range.x, part * Pt), k1 = min(range.y, (part + 1) * Pt);
    const int32_t *row = a.block_tables + (size_t)r.s * a.max_blocks;
    const float *kc = static_cast<const float *>(a.k_cache);
    const float *vc = static_cast<const float *>(a.v_cache);
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + ((size_t)i * a.Hq + kvh * G) * D);
    for (int c = threadIdx.x; c < G * D / 4; c += blockDim.x) qs[c / (D / 4)][c % (D / 4)] = q[c];
    float slope[G];
#pragma unroll
    for (int g = 0; g < G; ++g) slope[g] = a.slopes ? a.slopes[kvh * G + g] * kLog2e : 0.f;
    __syncthreads();

    const int e = lane & 7, sub = lane & 24;
    const int mine = 4 * e + (lane >> 3);  // this lane's key of a tile
    float m[G], l[G];                      // l: of this lane's keys
    Floats<kPer> acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int d = 0; d < kPer; ++d) acc[g].f[d] = 0.f;
    }
    for (int t0 = k0 + 32 * warp; t0 < k1; t0 += 32 * kWarps) {
        const int j = t0 + mine;
        unsigned long long off = 0;
        bool in = j < k1;
        if (in) {
            const int blk = row[j / B];
            if (blk < 0 || blk >= a.N) {
                set_error(a.err, PA_DEVERR_BAD_BLOCK);
                in = false;
            } else {
                off = (((unsigned long long)blk * a.Hkv + kvh) * B + j % B) * D;
            }
        }
        const unsigned have = __ballot_sync(0xffffffffu, in);
        // partial dots of key 4 u + lane / 8, over this lane's chunks of the row
        float dot[G][8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float *k = kc + __shfl_sync(0xffffffffu, off, sub + u);
            const bool there = have >> (sub + u) & 1;
            float4 x[kChunks];
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                x[c] = there ? *(reinterpret_cast<const float4 *>(k) + 8 * c + e) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const float4 y = qs[g][8 * c + e];
                    s = fmaf(x[c].x, y.x, s);
                    s = fmaf(x[c].y, y.y, s);
                    s = fmaf(x[c].z, y.z, s);
                    s = fmaf(x[c].w, y.w, s);
                }
                dot[g][u] = s;
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // lane e of eight ends with the sum of their dot[g][e]
#pragma unroll
            for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
                for (int u = 0; u < w; ++u) {
                    const float send = e & w ? dot[g][u] : dot[g][u + w];
                    const float keep = e & w ? dot[g][u + w] : dot[g][u];
                    dot[g][u] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
            float z = -INFINITY;
            if (in) {
                z = dot[g][0] * a.scale;
                if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
                z = z * kLog2e - slope[g] * fabsf((float)(r.pos - j));
            }
            if (a.ws_logits && j < k1) a.ws_logits[((size_t)r.s * a.Hq + kvh * G + g) * cap + j] = z;
            const float mn = fmaxf(m[g], warp_max(z));
            const float mu = mn == -INFINITY ? 0.f : mn;
            const float al = ex2(m[g] - mu);  // 0 while m is -inf
            const float p = ex2(z - mu);
            l[g] = l[g] * al + p;
            m[g] = mn;
#pragma unroll
            for (int d = 0; d < kPer; ++d) acc[g].f[d] *= al;
            ps[warp][g][mine] = p;
        }
        __syncwarp();
        // eight rows of V in flight; keys without a row (weight 0) load none
        for (int v0 = 0; v0 < min(32, k1 - t0); v0 += 8) {
            Floats<kPer> v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int owner = (u & 3) * 8 + (v0 + u) / 4;
                const float *x = vc + __shfl_sync(0xffffffffu, off, owner);
                if (have >> owner & 1) {
                    v[u] = *reinterpret_cast<const Floats<kPer> *>(x + lane * kPer);
                } else {
#pragma unroll
                    for (int d = 0; d < kPer; ++d) v[u].f[d] = 0.f;
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float p = ps[warp][g][v0 + u];
#pragma unroll
                    for (int d = 0; d < kPer; ++d) acc[g].f[d] = fmaf(p, v[u].f[d], acc[g].f[d]);
                }
        }
        __syncwarp();
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], o);
        if (lane == 0) ml[warp][g] = make_float2(m[g], l[g]);
        accs[warp][g][lane] = acc[g];
    }
    __syncthreads();
    for (int g = warp; g < G; g += kWarps) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w][g].x);
        const float mu = M == -INFINITY ? 0.f : M;
        Floats<kPer> o;
#pragma unroll
        for (int d = 0; d < kPer; ++d) o.f[d] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float t = ex2(ml[w][g].x - mu);
            L = fmaf(t, ml[w][g].y, L);
            const Floats<kPer> x = accs[w][g][lane];
#pragma unroll
            for (int d = 0; d < kPer; ++d) o.f[d] = fmaf(t, x.f[d], o.f[d]);
        }
        const size_t at = ((size_t)i * a.Hq + kvh * G + g) * a.max_parts + part;
        if (p0 == p1) {
#pragma unroll
            for (int d = 0; d < kPer; ++d) o.f[d] = L != 0.f ? o.f[d] / L : 0.f;
            *reinterpret_cast<Floats<kPer> *>(out + g * D + lane * kPer) = o;
        } else {
            *reinterpret_cast<Floats<kPer> *>(a.ws_acc + at * D + lane * kPer) = o;
        }
        if ((p0 != p1 || a.ws_logits) && lane == 0) *reinterpret_cast<float2 *>(a.ws_ml + 2 * at) = make_float2(M, L);
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

template <int D>
cudaError_t launch_rows_t(const ScoredArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)((long long)a.T * a.Hkv), (unsigned)a.max_parts);
    switch (a.Hq / a.Hkv) {
        case 1: scored_rows_kernel<D, 1><<<grid, kWarps * 32, 0, st>>>(a); break;
        case 2: scored_rows_kernel<D, 2><<<grid, kWarps * 32, 0, st>>>(a); break;
        case 4: scored_rows_kernel<D, 4><<<grid, kWarps * 32, 0, st>>>(a); break;
        case 8: scored_rows_kernel<D, 8><<<grid, kWarps * 32, 0, st>>>(a); break;
        default: return cudaErrorNotSupported;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scored_rows(const ScoredArgs &a, cudaStream_t st) {
    if (a.query_start) {
        scored_check_kernel<<<1, 1024, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.D == 64) return launch_rows_t<64>(a, st);
    if (a.D == 128) return launch_rows_t<128>(a, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
