// pa_attend8_plan.cu -- the work list of long chunks over the 8-bit cache: one entry
// per (sequence, group of 128-row tiles), those with the most steps first; or the line of
// all entries' steps, and where each CTA's stretch of it starts.
#include "pa_attend8.cuh"

namespace pa {

namespace {

__global__ void __launch_bounds__(1024) attend8_plan_kernel(const Attend8Args a, int groups) {
    constexpr int kBins = 1024;  // longer entries share the last bin
    __shared__ int hist[kBins], start[kBins], warp_sums[32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    griddep_wait();
    const int tid = threadIdx.x, G = a.Hq / a.Hkv;
    hist[tid] = 0;
    bool ok = true;
    for (int s = tid; s < a.S; s += 1024) ok = ok && order_ok(a, s);
    ok = __syncthreads_and(ok);
    if (!ok && tid == 0) {
        set_error(a.err, PA_DEVERR_BAD_LEN);
        a.hdr[0] = 0;
    }
    if (a.units) {
        for (int x = tid; x < a.units; x += 1024) {
            a.notes[x] = make_int4(0, 0, 0, 0);
            if (!ok) a.starts[x] = make_int4(0, 0, 0, 0);
        }
        if (!ok) return;
        // the line: a thread's entries (as if their steps came before any head's), and where they begin
        const int all = a.S * groups, per = (all + 1023) / 1024, e0 = min(all, tid * per), e1 = min(all, e0 + per);
        auto steps = [&](int e, bool flag) {
            const Seq8 q = seq_of(a, e / groups, flag && e % groups == 0);
            const int r0 = e % groups * 128 * a.tiles;
            return r0 < q.n * G ? span_of(a, q, r0).st.count : 0;
        };
        long long own = 0;
        for (int e = e0; e < e1; ++e) own += steps(e, true);
        long long incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if ((tid & 31) >= o) incl += u;
        }
        __shared__ long long sums[32];
        if ((tid & 31) == 31) sums[tid >> 5] = incl;
        __syncthreads();
        long long total = 0, at = incl - own;
        for (int w = 0; w < 32; ++w) {
            total += sums[w];
            if (w < tid >> 5) at += sums[w];
        }
        total *= a.Hkv;
        const long long share = max((long long)kLeastSteps8, (total + a.units - 1) / a.units);
        if (tid == 0) {
            a.hdr[0] = 1;
            a.hdr[1] = (int)share;
        }
        for (int e = e0; e < e1; ++e) {
            const int count = steps(e, false);
            const long long u0 = at * a.Hkv, u1 = u0 + (long long)count * a.Hkv;
            for (long long x = (u0 + share - 1) / share; x * share < u1; ++x) {
                const long long in = x * share - u0;
                a.starts[x] = make_int4(e, (int)(in / count), (int)(in % count), (int)min(share, total - x * share));
            }
            at += count;
        }
        for (long long x = (total + share - 1) / share + tid; x < a.units; x += 1024) a.starts[x] = make_int4(0, 0, 0, 0);
        return;
    }
    if (!ok) return;
    // the entry's bin, or -1 if its sequence has no rows there
    auto bin_of = [&](int s, int group, bool flag) {
        const Seq8 q = seq_of(a, s, flag);
        const int r0 = group * 128 * a.tiles;
        return r0 < q.n * G ? min(span_of(a, q, r0).st.count, kBins - 1) : -1;
    };
    const long long entries = (long long)a.S * groups;
    for (long long e = tid; e < entries; e += 1024) {
        const int s = (int)(e / groups), group = (int)(e % groups);
        const int bin = bin_of(s, group, group == 0);
        if (bin >= 0) atomicAdd(&hist[bin], 1);
    }
    __syncthreads();
    const int total = scan_bins_desc(hist, start, kBins - 1, kBins, warp_sums);
    if (tid == 0) {
        a.hdr[0] = total;
        a.hdr[1] = 0;
    }
    for (long long e = tid; e < entries; e += 1024) {
        const int s = (int)(e / groups), group = (int)(e % groups);
        const int bin = bin_of(s, group, false);
        if (bin >= 0) a.list[atomicAdd(&start[bin], 1)] = make_int4(s, group, 0, 0);
    }
}

}  // namespace

cudaError_t launch_attend8_plan(const Attend8Args &a, cudaStream_t st) {
    const int rows = 128 * a.tiles;
    const int groups = (int)(((long long)a.max_query_len * (a.Hq / a.Hkv) + rows - 1) / rows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend8_plan_kernel, a, groups);
}

}  // namespace pa
