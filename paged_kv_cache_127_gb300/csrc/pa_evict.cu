// pa_evict.cu -- eviction by summed attention weights: which tokens each KV head
// keeps, and their copy to fresh blocks.
//
// Selection, one cluster of CTAs per (sequence, KV head): of the n = len - recent
// older tokens the m = keep - recent with the largest sums.  Sums become 32-bit keys
// whose unsigned order is theirs (NaN lowest, -0 as +0).  Each CTA holds a slice of
// the keys in shared memory; the m-th largest key is found by radix selection, a
// digit of 11 or 10 bits a pass, over the cluster's histograms (read through distributed shared
// memory).  A token is kept if its key is larger, or equal and among the first
// `want` equal ones in index order, or if it is recent.  With G(j) larger and E(j)
// equal keys before token j, its new position is G(j) + min(E(j), want), a recent
// one's m + j - n: counts of larger and equal keys by segment give them all.  Each new
// place gets the token's cache slot (the move list) and its sum.
//
// Copy: 16 bytes of a K and a V row per thread and row, several rows in flight.
//
// Bound: HBM for a batch (the kept rows, read and written); latency for one sequence.
// Measured: 64 sequences of 2500 to 4096 tokens cut to 2048 (8 KV heads, D 128, bf16) 184 us, of which the
// selection 20 and the copy 162 (6.3 TB/s; floor 159); one of 32768 tokens cut to 8192 (D 64) 14 + 10 us.
#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_scored.h"

namespace cg = cooperative_groups;

namespace pa {

namespace {

constexpr int kMaxSlice = 48 * 1024;  // keys of a slice kept in shared memory

// Unsigned order of the keys = order of the sums; NaN below everything.
__device__ __forceinline__ uint32_t sum_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of v over the block (all threads call).
template <int kThreads>
__device__ __forceinline__ int block_scan(int v, int *warp_sums) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[wid] = incl;
    __syncthreads();
    static_assert(kThreads / 32 <= 32, "one lane a warp");
    const int base = __reduce_add_sync(0xffffffffu, lane < wid && lane < kThreads / 32 ? warp_sums[lane] : 0);
    return base + incl - v;
}

// Radix digits, from the top.  11 bits first: sums are positive numbers of a few
// octaves, whose top 8 bits (sign and 7 of the exponent) would fall into a handful of bins
// that every thread of the block then adds to.
constexpr int kBins = 2048;

// kFit: the cluster's slices hold every key in shared memory; else the keys are
// read from the sums again in each pass.  kCluster: more than one CTA a (sequence, head).
template <bool kFit, bool kCluster, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int lb) {
    constexpr int kWarps = kSelThreads / 32;
    extern __shared__ uint32_t keys[];          // kFit: this CTA's slice
    __shared__ alignas(16) int hist[2][kBins];  // counts, alternating between passes
    __shared__ int warp_sums[kWarps];
    __shared__ int2 found[kWarps];  // larger and equal keys of each warp's segment
    __shared__ int2 slice_total;
    __shared__ uint32_t s_key;
    __shared__ int s_want, s_done;
    cg::cluster_group cluster = cg::this_cluster();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int C = kCluster ? (int)cluster.num_blocks() : 1, rank = kCluster ? (int)cluster.block_rank() : 0;
    auto sync_all = [&] {
        if constexpr (kCluster) cluster.sync();
        else __syncthreads();
    };
    const int pair = blockIdx.x / C, s = pair / a.Hkv, h = pair % a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = a.max_blocks * a.B;
    int len = a.lens[s], keep = a.keep_lens[s];
    const int row = a.sum_rows ? a.sum_rows[s] : s;
    const bool first = tid == 0 && rank == 0;
    if (len < 0 || len > cap || keep < 0) {
        if (first && h == 0) set_error(a.err, PA_DEVERR_BAD_LEN);
        len = len < 0 ? 0 : (len > cap ? cap : len);
        if (keep < 0) keep = len;
    }
    const bool bad_row = row < 0 || row >= a.sum_num_rows;
    if (bad_row) {
        if (first && h == 0) set_error(a.err, PA_DEVERR_BAD_ROW);
        keep = len;
    }
    const int now = min(len, keep);
    if (first) {
        a.counts[pair] = len > keep ? keep : 0;
        if (h == 0) a.new_lens[s] = now;
    }
    if (bad_row) return;  // the whole cluster
    const float *in = a.sums + ((size_t)row * a.Hkv + h) * a.sum_cols;
    float *out = a.sums_out + ((size_t)row * a.Hkv + h) * a.sum_cols;
    if (len <= keep) {
        for (int j = rank * kSelThreads + tid; j < a.sum_cols; j += C * kSelThreads) out[j] = j < now ? in[j] : 0.f;
        return;  // the whole cluster
    }
    const int recent = min(a.recent, keep);
    const int n = len - recent, m = keep - recent;  // m < n
    const int slice = ((n + C - 1) / C + 3) & ~3;
    const int j0 = min(n, rank * slice), count = min(n, j0 + slice) - j0;  // this CTA's older tokens
    const float *mine = in + j0;
    if (kFit) {
        const int whole = count & ~3;  // j0 is a multiple of 4 unless count is 0
        for (int j = 4 * tid; j < whole; j += 4 * kSelThreads) {
            const float4 x = *reinterpret_cast<const float4 *>(mine + j);
            *reinterpret_cast<uint4 *>(keys + j) = make_uint4(sum_key(x.x), sum_key(x.y), sum_key(x.z), sum_key(x.w));
        }
        if (tid < count - whole) keys[whole + tid] = sum_key(mine[whole + tid]);
    }
    auto key_at = [&](int j) { return kFit ? keys[j] : sum_key(mine[j]); };
    for (int b = tid; b < kBins; b += kSelThreads) hist[0][b] = 0;
    __syncthreads();
    // the m-th largest key, a digit at a time; `want` of the keys that share the prefix so far
    uint32_t prefix = 0, known = 0xffffffffu;  // a key counts as equal if its `known` bits are
    int want = m;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        if (m == 0) break;
        constexpr int kPer = kBins / kSelThreads;
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass < 2 ? 11 : 10;
        const uint32_t mask = (1u << digits) - 1u;
        const uint32_t high = pass == 0 ? 0u : 0xffffffffu << (shift + digits);
        int *mh = hist[pass & 1];
        auto add = [&](uint32_t k) {
            if ((k & high) == prefix) atomicAdd(&mh[k >> shift & mask], 1);
        };
        int j = 0;
        if (kFit)
            for (; j + 4 * kSelThreads <= count; j += 4 * kSelThreads) {
                const uint4 k = *reinterpret_cast<const uint4 *>(keys + j + 4 * tid);
                add(k.x);
                add(k.y);
                add(k.z);
                add(k.w);
            }
        for (j += tid; j < count; j += kSelThreads) add(key_at(j));
        sync_all();
        // bins from the largest down, kPer a thread: the one that holds the want-th key
        int v[kPer], sum = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = 0;
        auto add_bins = [&](const int *counts) {
            const int2 *x = reinterpret_cast<const int2 *>(counts + kBins - kPer * (tid + 1));
#pragma unroll
            for (int e = 0; e < kPer / 2; ++e) {
                const int2 b = x[kPer / 2 - 1 - e];
                v[2 * e] += b.y;
                v[2 * e + 1] += b.x;
            }
        };
        if constexpr (kCluster) {
#pragma unroll 4
            for (int c = 0; c < C; ++c) add_bins(cluster.map_shared_rank(mh, c));
        } else {
            add_bins(mh);
        }
        static_assert(kPer % 2 == 0, "pairs of bins");
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum += v[e];
        // the other counts, which the cluster read before the sync above, for the next pass
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) reinterpret_cast<int2 *>(hist[~pass & 1])[tid + e * kSelThreads] = make_int2(0, 0);
        int before = block_scan<kSelThreads>(sum, warp_sums);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            if (before < want && want <= before + v[e]) {
                s_key = prefix | (uint32_t)(kBins - 1 - kPer * tid - e) << shift;
                s_want = want - before;
                s_done = want - before == v[e];  // every key of the bin is kept: its lower bits do not matter
            }
            before += v[e];
        }
        __syncthreads();
        prefix = s_key;
        want = s_want;
        known = mask << shift | high;
        const int done = s_done;
        __syncthreads();
        if (done) break;  // the whole cluster alike
    }
    // larger and equal keys: each warp counts a segment of the slice, 32 keys at a time
    const int seg = (((count + kWarps - 1) / kWarps) + 31) & ~31;
    const int w0 = min(count, warp * seg), w1 = min(count, w0 + seg);
    int larger = 0, equal = 0;
    for (int j = w0 + lane; j - lane < w1 && m > 0; j += 32) {
        const uint32_t k = j < w1 ? key_at(j) & known : 0u;
        larger += __popc(__ballot_sync(0xffffffffu, j < w1 && k > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, j < w1 && k == prefix));
    }
    if (lane == 0) found[warp] = make_int2(larger, equal);
    __syncthreads();
    const int2 mine_of = lane < kWarps ? found[lane] : make_int2(0, 0);
    larger = __reduce_add_sync(0xffffffffu, lane < warp ? mine_of.x : 0);
    equal = __reduce_add_sync(0xffffffffu, lane < warp ? mine_of.y : 0);
    if (tid == kSelThreads - 1) slice_total = make_int2(larger + found[kWarps - 1].x, equal + found[kWarps - 1].y);
    sync_all();
    if constexpr (kCluster)
        for (int c = 0; c < rank; ++c) {
            const int2 t = *cluster.map_shared_rank(&slice_total, c);
            larger += t.x;
            equal += t.y;
        }
    // the kept tokens' old positions, at their new ones
    int *list = a.list + (size_t)pair * cap;
    for (int j = w0 + lane; j - lane < w1 && m > 0; j += 32) {
        const uint32_t k = j < w1 ? key_at(j) & known : 0u;
        const bool gt = j < w1 && k > prefix, eq = j < w1 && k == prefix;
        const unsigned gts = __ballot_sync(0xffffffffu, gt), eqs = __ballot_sync(0xffffffffu, eq);
        const unsigned below = (1u << lane) - 1u;
        const int g = larger + __popc(gts & below), e = equal + __popc(eqs & below);
        if (gt || (eq && e < want)) list[g + min(e, want)] = j0 + j;
        larger += __popc(gts);
        equal += __popc(eqs);
    }
    for (int i = rank * kSelThreads + tid; i < recent; i += C * kSelThreads) list[m + i] = n + i;
    // The copy's blocks may come now: earlier they would hold registers that this grid's CTAs need.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    sync_all();  // the list is complete, and the keys have been read
    // sums to their new places, and cache slots in place of positions.  A token never moves up, so
    // with sums_out == sums a tile of places is read before any of it is written.
    constexpr int kU = 4;
    const int32_t *table = a.tables + (size_t)s * a.max_blocks;
    const int tile = C * kSelThreads * kU;
    const bool in_place = in == out;
    for (int t0 = 0; t0 < keep; t0 += tile) {
        float x[kU];
        int slot[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = t0 + (u * C + rank) * kSelThreads + tid;
            slot[u] = -1;
            if (i < keep) {
                const int p = list[i];
                x[u] = in[p];
                const int tb = lb >= 0 ? p >> lb : p / a.B, b = table[tb];
                if (b >= 0 && b < a.N) slot[u] = b * a.B + (p - tb * a.B);
                else set_error(a.err, PA_DEVERR_BAD_BLOCK);
            }
        }
        if (in_place) sync_all();
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = t0 + (u * C + rank) * kSelThreads + tid;
            if (i < keep) {
                out[i] = x[u];
                list[i] = slot[u];
            }
        }
    }
    for (int j = keep + rank * kSelThreads + tid; j < a.sum_cols; j += C * kSelThreads) out[j] = 0.f;
}

// Copy of the listed rows.  A block takes `tiles` tiles of rows; in a tile a thread moves
// 16-byte chunk c of kRowsInFlight rows, K and V, all loads before the stores, and has read
// the next tile's slots by then.  lb: log2 of the block size, or -1.
constexpr int kMoveThreads = 256;
constexpr int kRowsInFlight = 4;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int chunks, int lb, int tiles) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int pair = blockIdx.y, s = pair / a.Hkv, h = pair % a.Hkv;
    const int width = min(chunks, kMoveThreads), per = kMoveThreads / width;  // threads of a row, rows side by side
    const int rows = per * kRowsInFlight;                                     // of a tile
    int r = blockIdx.x * rows * tiles + (int)threadIdx.x / width;
    const int count = a.counts[pair];
    const int end = min(count, (int)(blockIdx.x + 1) * rows * tiles);
    if (r >= end || (int)threadIdx.x >= width * per) return;
    const int cap = a.max_blocks * a.B;
    const int32_t *to = a.new_tables + (size_t)s * a.max_blocks;
    const int *list = a.list + (size_t)pair * cap;
    uint4 *kc = static_cast<uint4 *>(a.k_cache), *vc = static_cast<uint4 *>(a.v_cache);
    auto block_of = [&](int x) { return lb >= 0 ? x >> lb : x / a.B; };
    int slot[kRowsInFlight], tb[kRowsInFlight];
    auto fetch = [&](int r) {
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
            slot[u] = -1;
            if (r + u * per < end) {
                slot[u] = list[r + u * per];
                tb[u] = to[block_of(r + u * per)];
            }
        }
    };
    fetch(r);
    for (; r < end; r += rows) {
        int src[kRowsInFlight], dst[kRowsInFlight];  // rows of the cache
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
            src[u] = -1;
            if (slot[u] < 0) continue;
            if (tb[u] < 0 || tb[u] >= a.N) {
                set_error(a.err, PA_DEVERR_BAD_BLOCK);
                continue;
            }
            const int fb = block_of(slot[u]), at = r + u * per;
            src[u] = (fb * a.Hkv + h) * a.B + (slot[u] - fb * a.B);
            dst[u] = (tb[u] * a.Hkv + h) * a.B + (at - block_of(at) * a.B);
        }
        if (r + rows >= end) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        fetch(r + rows);
        for (int c = (int)threadIdx.x % width; c < chunks; c += kMoveThreads) {
            uint4 k[kRowsInFlight], v[kRowsInFlight];
#pragma unroll
            for (int u = 0; u < kRowsInFlight; ++u)
                if (src[u] >= 0) {
                    k[u] = __ldcs(kc + (size_t)src[u] * chunks + c);
                    v[u] = __ldcs(vc + (size_t)src[u] * chunks + c);
                }
#pragma unroll
            for (int u = 0; u < kRowsInFlight; ++u)
                if (src[u] >= 0) {
                    kc[(size_t)dst[u] * chunks + c] = k[u];
                    vc[(size_t)dst[u] * chunks + c] = v[u];
                }
        }
    }
}

template <bool kFit, bool kCluster, int kSelThreads>
cudaError_t launch_select(const EvictArgs &a, int C, int lb, size_t smem, cudaStream_t st) {
    static std::atomic<int> configured[kMaxLaunchDevices];
    int one = 0;
    const cudaError_t e = per_device_value(configured, &one, [](int, int *v) {
        *v = 1;
        return cudaFuncSetAttribute(evict_select_kernel<kFit, kCluster, kSelThreads>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kFit ? kMaxSlice * 4 : 0);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.S * a.Hkv * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<kFit, kCluster, kSelThreads>, a, lb);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st) {
    if (a.S == 0) return cudaSuccess;
    const int cap = a.max_blocks * a.B, pairs = a.S * a.Hkv;
    // CTAs per (sequence, KV head): while two CTAs an SM are not filled and a slice stays above 1024
    // keys, and as many as the keys need to fit in shared memory, at most 8 (a portable cluster)
    int C = 1;
    while (C < 8 && ((pairs * C < 2 * 152 && cap / C >= 2048) || cap / C > kMaxSlice - 8)) C *= 2;
    const int slice = (((cap + C - 1) / C) + 7) & ~3;
    const bool fit = slice <= kMaxSlice;
    const int lb = (a.B & (a.B - 1)) == 0 ? __builtin_ctz((unsigned)a.B) : -1;  // log2 of the block size, or -1
    // Small CTAs when every SM holds several (less of the fixed work a warp does), large ones when a
    // pair's chain of steps is what takes the time.
    cudaError_t e = !fit      ? launch_select<false, true, 1024>(a, C, lb, 0, st)
                    : C > 1   ? launch_select<true, true, 1024>(a, C, lb, (size_t)slice * 4, st)
                    : pairs >= 152 ? launch_select<true, false, 256>(a, C, lb, (size_t)slice * 4, st)
                                   : launch_select<true, false, 1024>(a, C, lb, (size_t)slice * 4, st);
    if (e != cudaSuccess) return e;
    // The copy wants the whole L1 for its loads in flight: left with the split that the selection's
    // shared memory asked for, it takes 208 us for 64 sequences instead of 168.
    static std::atomic<int> configured[kMaxLaunchDevices];
    int one = 0;
    e = per_device_value(configured, &one, [](int, int *v) {
        *v = 1;
        return cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxL1);
    });
    if (e != cudaSuccess) return e;
    const int chunks = a.row_bytes / 16;
    const int rows = kRowsInFlight * (chunks < kMoveThreads ? kMoveThreads / chunks : 1);
    cudaLaunchConfig_t cfg = {};
    // four tiles a block hide the next slots behind the copy, as long as they leave every SM its blocks
    const int tiles = (long long)pairs * (cap / rows) >= 4LL * 8 * 152 ? 4 : 1;
    cfg.gridDim = dim3((unsigned)((cap + rows * tiles - 1) / (rows * tiles)), (unsigned)pairs);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, a, chunks, lb, tiles);
}

}  // namespace pa
