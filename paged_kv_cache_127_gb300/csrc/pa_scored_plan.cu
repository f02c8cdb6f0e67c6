// pa_scored_plan.cu -- work list of the scored tensor-core decode.
//
// One CTA lists every (sequence, partition) that holds keys of the sequence's
// range, as (sequence, partition, first key, one past the last key), most 16-key
// chunks first (a counting sort), so that the persistent decode hands out big
// items before small ones.  Bit 30 of the partition marks an item that holds
// its sequence's whole range.  The first partition of the first
// min(S, ctas / groups) sequences is left out: decode CTA b takes it directly
// (sequence b / groups), before this list is complete.  The plan also
// resets the claim counters, writes the zero rows of empty ranges and flags bad
// lengths.
#include "pa_score.cuh"

namespace pa {

namespace {

constexpr int kBins = 1024;  // by chunk count, larger items binned together

__device__ __forceinline__ void zero_row(const ScoredArgs &a, int i) {
    const int n = a.Hq * a.D;
    uint4 *row = reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + (size_t)i * n * (a.out16 ? 2 : 4));
    for (int c = 0; c < n * (a.out16 ? 2 : 4) / 16; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
}

__global__ void __launch_bounds__(1024) scored_decode_plan_kernel(const ScoredArgs a) {
    __shared__ int hist[kBins];
    __shared__ int start[kBins];
    __shared__ int warp_sums[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, Pt = a.partition_size, cap = a.max_blocks * a.B;
    const int groups = a.Hkv / a.head_group;
    const int nstatic = min(a.S, a.ctas / groups);
    for (int i = tid; i < kBins; i += blockDim.x) hist[i] = 0;
    if (tid == 0) {
        a.plan_hdr[1] = 0;
        a.plan_hdr[2] = 0;
    }
    __syncthreads();
    for (int s = tid; s < a.S; s += blockDim.x) {
        const int len = a.context_lens[s];
        if (len < 0 || len > cap) set_error(a.err, PA_DEVERR_BAD_LEN);
        const RowOf r = row_of(a, s, cap);
        const int2 k = row_range(a, s, r.pos, r.len);
        if (k.x >= k.y) {
            zero_row(a, s);
            continue;
        }
        const int p0 = k.x / Pt, p1 = (k.y - 1) / Pt;
        for (int p = s < nstatic ? p0 + 1 : p0; p <= p1; ++p) {
            const int lo = max(k.x, p * Pt), hi = min(k.y, (p + 1) * Pt);
            atomicAdd(&hist[min((hi - (lo & ~15) + 15) >> 4, kBins - 1)], 1);
        }
    }
    __syncthreads();
    const int total = scan_bins_desc(hist, start, kBins - 1, kBins, warp_sums);
    if (tid == 0) a.plan_hdr[0] = total * groups;
    for (int s = tid; s < a.S; s += blockDim.x) {
        const RowOf r = row_of(a, s, cap);
        const int2 k = row_range(a, s, r.pos, r.len);
        if (k.x >= k.y) continue;
        const int p0 = k.x / Pt, p1 = (k.y - 1) / Pt;
        for (int p = s < nstatic ? p0 + 1 : p0; p <= p1; ++p) {
            const int lo = max(k.x, p * Pt), hi = min(k.y, (p + 1) * Pt);
            const int at = atomicAdd(&start[min((hi - (lo & ~15) + 15) >> 4, kBins - 1)], 1);
            a.plan_list[at] = make_int4(s, p | (p0 == p1 ? kWholeRange : 0), lo, hi);
        }
    }
}

}  // namespace

cudaError_t launch_scored_decode_plan(const ScoredArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_decode_plan_kernel, a);
}

}  // namespace pa
