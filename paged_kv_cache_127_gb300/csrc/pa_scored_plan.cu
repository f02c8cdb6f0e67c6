// pa_scored_plan.cu -- work lists of the scored tensor-core kernels.
//
// Decode: one CTA lists the pieces of every sequence's range (piece_of), as (sequence,
// piece, first key, one past the last key), most 16-key chunks first (a counting
// sort), so that the persistent decode hands out big items before small ones.
// Bit 30 of the piece marks an item that holds its sequence's whole range.  The
// first piece of the first min(S, ctas / groups) sequences is left out: decode CTA
// b takes it directly (sequence b / groups), before this list is complete.  Left to
// choose, the plan widens the other pieces while the batch still has enough of
// them: the host sees only the batch's shape, the plan its lengths, and longer pieces
// mean fewer partials (32 sequences of 8192-32768 tokens: 442 us with pieces of 256,
// 412 with 512, 397 with 1024; of 800 tokens: 26 us with 256, 34 with 512).  The plan also
// resets the claim counters, writes the zero rows of empty ranges and flags bad
// lengths.  Bound: latency; 7 to 9 us for 64 to 256 sequences, of which the decode's first items hide some.
#include <climits>

#include "pa_score.cuh"

namespace pa {

namespace {

constexpr int kBins = 1024;     // by chunk count, larger items binned together
constexpr int kMaxPiece = 1024;  // keys of a widened decode piece, at most (measured: 2048 is no faster)

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
    const int tid = threadIdx.x, size = a.partition_size, cap = a.max_blocks * a.B;
    const int groups = a.Hkv / a.head_group;
    const int nstatic = min(a.S, a.ctas / groups);
    for (int i = tid; i < kBins; i += blockDim.x) hist[i] = 0;
    __shared__ int merges;  // sequences whose range lies in several pieces
    __shared__ int counts[2];  // pieces of twice and four times the size
    if (tid == 0) {
        a.plan_hdr[1] = 0;
        merges = counts[0] = counts[1] = 0;
    }
    __syncthreads();
    int wide = size;
    if (a.widen) {
        int n2 = 0, n4 = 0;
        for (int s = tid; s < a.S; s += blockDim.x) {
            const RowOf r = row_of(a, s, cap);
            const int2 k = row_range(a, s, r.pos, r.len);
            if (k.x >= k.y) continue;
            n2 += pieces_of(k, size, 2 * size);
            n4 += pieces_of(k, size, 4 * size);
        }
        n2 = __reduce_add_sync(0xffffffffu, n2);
        n4 = __reduce_add_sync(0xffffffffu, n4);
        if ((tid & 31) == 0 && n2 > 0) {
            atomicAdd(&counts[0], n2);
            atomicAdd(&counts[1], n4);
        }
        __syncthreads();
        // at least 1.5 items a CTA, 3 for pieces of 1024 and more (whose ends leave CTAs idle longer)
        auto enough = [&](int count, int to) { return 2LL * count * groups >= (to >= 1024 ? 6LL : 3LL) * a.ctas; };
        if (enough(counts[0], 2 * size) && 2 * size <= kMaxPiece) {
            wide = 2 * size;
            if (enough(counts[1], 4 * size) && 4 * size <= kMaxPiece) wide = 4 * size;
        }
    }
    for (int s = tid; s < a.S; s += blockDim.x) {
        const int len = a.context_lens[s];
        if (len < 0 || len > cap) set_error(a.err, PA_DEVERR_BAD_LEN);
        const RowOf r = row_of(a, s, cap);
        const int2 k = row_range(a, s, r.pos, r.len);
        if (k.x >= k.y) {
            zero_row(a, s);
            continue;
        }
        const int np = pieces_of(k, size, wide);
        if (np > 1) a.merge_list[atomicAdd(&merges, 1)] = make_int4(s, 0, np - 1, 0);
        for (int i = s < nstatic ? 1 : 0; i < np; ++i) {
            const int2 p = piece_of(k, size, wide, i);
            atomicAdd(&hist[min((p.y - (p.x & ~15) + 15) >> 4, kBins - 1)], 1);
        }
    }
    __syncthreads();
    const int total = scan_bins_desc(hist, start, kBins - 1, kBins, warp_sums);
    if (tid == 0) {
        a.plan_hdr[0] = total * groups;
        a.plan_hdr[2] = merges;
        a.plan_hdr[3] = wide;
    }
    for (int s = tid; s < a.S; s += blockDim.x) {
        const RowOf r = row_of(a, s, cap);
        const int2 k = row_range(a, s, r.pos, r.len);
        if (k.x >= k.y) continue;
        const int np = pieces_of(k, size, wide);
        for (int i = s < nstatic ? 1 : 0; i < np; ++i) {
            const int2 p = piece_of(k, size, wide, i);
            const int at = atomicAdd(&start[min((p.y - (p.x & ~15) + 15) >> 4, kBins - 1)], 1);
            a.plan_list[at] = make_int4(s, i | (np == 1 ? kWholeRange : 0), p.x, p.y);
        }
    }
}

// Chunk calls.  An entry is a row block of a sequence -- the tcgen05 path's group
// of one or two 128-row tiles, or the mma.sync path's 16 or 32 rows -- and, on
// the mma.sync path, a partition: (sequence, block, lo, hi) or (sequence,
// partition | block << 16, lo, hi), with the keys [lo, hi) that some row of the
// block sees; most keys first.  Two passes over the blocks, counting and
// placing, a thread each.  With key_begin or key_end the blocks' spans come
// first, a warp per block into shared memory (zeroing empty rows on the way); calls of
// more than kSpanCache blocks take a warp per block in both passes instead.  On the mma.sync path
// the rows whose range lies in several partitions are listed for the merge.
// An entry of the tcgen05 path is marked (kHoles) unless one of its rows sees all of [lo, hi), or each row's range
// meets that of the last one before it that sees anything: then its rows together see every key of [lo, hi).
// plan_hdr[0] = -1 when query_start is not non-decreasing within [0, T].
constexpr int kSeqCache = 2048;
constexpr int kSpanCache = 2048;

// A row block: its first token and one past its last (none: an empty range) of the sequence's chunk, and the
// sequence's first row, tokens before the chunk and length.
struct ChunkBlock {
    int t0, t1, q0, before, len;
};

// Whether the range of some token of a block does not meet that of the last one before it that sees
// anything.  Whole warp.  (Out of line: inlined it takes the registers of the masks in flight, 10.1 -> 10.9 us for
// 16 x 512 rows.)
__device__ __noinline__ bool ranges_apart(const ScoredArgs &a, ChunkBlock k0, int lane) {
    int2 last = make_int2(0, 0);
    bool apart = false;
    for (int b = k0.t0; b < k0.t1; b += 32) {
        const int t = b + lane;
        const int2 k = t < k0.t1 ? row_range(a, k0.q0 + t, k0.before + t, k0.len) : make_int2(0, 0);
        const unsigned live = __ballot_sync(0xffffffffu, k.x < k.y);
        const int from = 31 - __clz(live & ((1u << lane) - 1u)), top = 31 - __clz(live);
        const int x = __shfl_sync(0xffffffffu, k.x, from & 31), y = __shfl_sync(0xffffffffu, k.y, from & 31);
        const int2 prev = from >= 0 ? make_int2(x, y) : last;
        apart |= k.x < k.y && prev.x < prev.y && max(k.x, prev.x) > min(k.y, prev.y);
        const int2 end = make_int2(__shfl_sync(0xffffffffu, k.x, top & 31), __shfl_sync(0xffffffffu, k.y, top & 31));
        if (live) last = end;
    }
    return __any_sync(0xffffffffu, apart);
}

__global__ void __launch_bounds__(1024) scored_chunk_plan_kernel(const ScoredArgs a) {
    __shared__ int hist[kBins];
    __shared__ int start[kBins];
    __shared__ int warp_sums[32];
    __shared__ int qs_cache[kSeqCache + 1];
    __shared__ int len_cache[kSeqCache];
    __shared__ int2 spans[kSpanCache];
    __shared__ int merges;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31;
    const int G = a.Hq / a.Hkv, cap = a.max_blocks * a.B;
    const int rows = a.umma_rows > 0 ? a.umma_rows : 16 * a.row_warps;  // query rows of a block
    const int tokens = rows / G;                                        // its tokens (G divides rows)
    const int Pt = a.umma_rows > 0 ? INT_MAX : a.partition_size;
    const int unit = a.umma_rows > 0 ? PA_CHUNK_UMMA_KEYS : 16;         // keys of a step
    const bool cached = a.S <= kSeqCache;
    const int blocks = (a.max_query_len + tokens - 1) / tokens;  // of a sequence, at most
    const unsigned all = (unsigned)a.S * (unsigned)blocks;       // bounded by the entry point
    const bool masks = a.key_begin || a.key_end;  // else the ranges follow from the positions, and none is empty
    const bool in_smem = masks && all <= kSpanCache;
    if (cached) {
        for (int s = tid; s <= a.S; s += blockDim.x) qs_cache[s] = a.query_start[s];
        for (int s = tid; s < a.S; s += blockDim.x) len_cache[s] = a.context_lens[s];
    }
    for (int i = tid; i < kBins; i += blockDim.x) hist[i] = 0;
    if (tid == 0) {
        a.plan_hdr[1] = 0;
        merges = 0;
    }
    __syncthreads();
    const int *qs = cached ? qs_cache : a.query_start;
    const int *lens = cached ? len_cache : a.context_lens;
    int bad = tid == 0 && (qs[0] < 0 || qs[a.S] > a.T);
    for (int s = tid; s < a.S; s += blockDim.x) bad |= qs[s] > qs[s + 1];
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            set_error(a.err, PA_DEVERR_BAD_LEN);
            a.plan_hdr[0] = -1;
            a.plan_hdr[2] = 0;
        }
        return;
    }
    for (int s = tid; s < a.S; s += blockDim.x) {
        const int len = lens[s], n = qs[s + 1] - qs[s];
        if (len < 0 || len > cap || n > len || n > a.max_query_len) set_error(a.err, PA_DEVERR_BAD_LEN);
    }
    // The row's sequence, or -1 (qs[s0] <= i, or s0 == 0; the row's sequence in [s0, s1)).
    auto seq_of = [&](int i) {
        int s0 = 0, s1 = a.S;
        while (s1 - s0 > 1) {
            const int mid = (s0 + s1) >> 1;
            if (qs[mid] <= i) s0 = mid; else s1 = mid;
        }
        const int n = qs[s0 + 1] - qs[s0], len = lens[s0], t = i - qs[s0];
        return t < 0 || t >= n || len < 0 || len > cap || n > len || n > a.max_query_len ? -1 : s0;
    };
    // Block b of the call.
    auto block_at = [&](unsigned b) {
        const int s = (int)(b / (unsigned)blocks), rb = (int)(b - (unsigned)s * (unsigned)blocks);
        const int q0 = qs[s], n = qs[s + 1] - q0, len = lens[s];
        ChunkBlock k{rb * tokens, min(n, (rb + 1) * tokens), q0, len - n, len};
        if (len < 0 || len > cap || n > len || n > a.max_query_len) k.t1 = 0;
        return k;
    };
    if (in_smem) {
        // A warp per block, the masks of kAhead blocks in flight (a thread per row, searching its sequence
        // and updating its block's span: 12.6 us for 16 x 512 rows, this 8.9, 10.1 with the marks).
        constexpr int kAhead = 4;
        for (unsigned b0 = tid >> 5; b0 < all; b0 += 32 * kAhead) {
            int lo[kAhead], hi[kAhead];
            unsigned covers = 0u;  // bit u: one of the lane's rows sees all of lo[u] .. hi[u]
#pragma unroll
            for (int u = 0; u < kAhead; ++u) lo[u] = INT_MAX, hi[u] = 0;
            for (int e = lane; e < tokens; e += 32) {
                int begin[kAhead], end[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const ChunkBlock k = block_at(min(b0 + 32u * u, all - 1));
                    const bool in = b0 + 32u * u < all && k.t0 + e < k.t1;
                    begin[u] = in && a.key_begin ? a.key_begin[k.q0 + k.t0 + e] : 0;
                    end[u] = in && a.key_end ? a.key_end[k.q0 + k.t0 + e] : INT_MAX;
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const ChunkBlock k = block_at(min(b0 + 32u * u, all - 1));
                    const int t = k.t0 + e, pos = k.before + t;
                    if (b0 + 32u * u >= all || t >= k.t1) continue;
                    const int x = max(max(0, begin[u]), a.window > 0 ? pos - a.window + 1 : 0);
                    const int y = min(k.len, a.key_end ? end[u] : pos + 1);
                    if (x < y) {
                        if (x <= lo[u] && y >= hi[u]) covers |= 1u << u;
                        else if (x < lo[u] || y > hi[u]) covers &= ~(1u << u);
                        lo[u] = min(lo[u], x);
                        hi[u] = max(hi[u], y);
                    } else {
                        zero_row(a, k.q0 + t);
                    }
                }
            }
            __syncwarp();
            unsigned look = 0u;  // blocks of which no row sees all
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int x = __reduce_min_sync(0xffffffffu, lo[u]), y = __reduce_max_sync(0xffffffffu, hi[u]);
                if (lane == 0 && b0 + 32u * u < all) spans[b0 + 32u * u] = make_int2(x, y);
                if (a.umma_rows > 0 && x < y && !__any_sync(0xffffffffu, lo[u] == x && hi[u] == y && (covers >> u & 1u)))
                    look |= 1u << u;
            }
            for (; look; look &= look - 1u) {
                const unsigned b = b0 + 32u * (unsigned)(__ffs(look) - 1);
                if (ranges_apart(a, block_at(b), lane) && lane == 0) spans[b].y |= kHoles;
            }
        }
        __syncthreads();
    }
    const bool arrays = masks && !in_smem;
    const unsigned first = arrays ? tid >> 5 : tid, stride = arrays ? 32 : 1024;
    const int l0 = arrays ? lane : 0, lstep = arrays ? 32 : 1;   // the lanes of a warp share a block's partitions
    for (int pass = 0; pass < 2; ++pass) {
        for (unsigned b = first; b < all; b += stride) {
            const int s = (int)(b / (unsigned)blocks), rb = (int)(b - (unsigned)s * (unsigned)blocks);
            const ChunkBlock at = block_at(b);
            if (at.t0 >= at.t1) continue;
            int2 k;
            int holes = 0;
            if (in_smem) {
                k = spans[b];
                holes = k.y & kHoles;
                k.y &= ~kHoles;
            } else if (!masks) {
                k.x = a.window > 0 ? max(0, at.before + at.t0 - a.window + 1) : 0;
                k.y = at.before + at.t1;
            } else {
                int lo = INT_MAX, hi = 0, longest = 0;
                for (int t = at.t0 + lane; t < at.t1; t += 32) {
                    const int2 r = row_range(a, at.q0 + t, at.before + t, at.len);
                    if (r.x < r.y) {
                        lo = min(lo, r.x);
                        hi = max(hi, r.y);
                        longest = max(longest, r.y - r.x);
                    } else if (pass == 0) {
                        zero_row(a, at.q0 + t);
                    }
                }
                k.x = __reduce_min_sync(0xffffffffu, lo);
                k.y = __reduce_max_sync(0xffffffffu, hi);
                if (a.umma_rows > 0 && pass == 1 && __reduce_max_sync(0xffffffffu, longest) < k.y - k.x)
                    holes = ranges_apart(a, at, lane) ? kHoles : 0;
            }
            if (k.x >= k.y) continue;
            const int p0 = k.x / Pt, p1 = (k.y - 1) / Pt;
            for (int p = p0 + l0; p <= p1; p += lstep) {
                const int lo = p == p0 ? k.x : p * Pt, hi = p == p1 ? k.y : (p + 1) * Pt;
                const int bin = min((hi - 1) / unit - lo / unit + 1, kBins - 1);
                if (pass == 0) {
                    atomicAdd(&hist[bin], 1);
                } else {
                    const int place = atomicAdd(&start[bin], 1);
                    a.plan_list[place] = make_int4(s | holes, a.umma_rows > 0 ? rb : p | rb << 16, lo, hi);
                }
            }
        }
        if (pass == 0 && a.umma_rows == 0 && a.max_parts > 1) {
            for (int i = tid; i < a.T; i += blockDim.x) {
                const int s = seq_of(i);
                if (s < 0) continue;
                const int n = qs[s + 1] - qs[s], len = lens[s], t = i - qs[s];
                const int2 k = row_range(a, i, len - n + t, len);
                if (k.x >= k.y) continue;
                const int p0 = k.x / Pt, p1 = (k.y - 1) / Pt;
                if (p0 != p1) a.merge_list[atomicAdd(&merges, 1)] = make_int4(i, p0, p1, 0);
            }
        }
        __syncthreads();
        if (pass == 0) {
            const int total = scan_bins_desc(hist, start, kBins - 1, kBins, warp_sums);
            if (tid == 0) {
                a.plan_hdr[0] = total;
                a.plan_hdr[2] = merges;
            }
        }
    }
}

}  // namespace

cudaError_t launch_scored_chunk_plan(const ScoredArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_chunk_plan_kernel, a);
}

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
