// pa_attend8_mma.cuh -- decode and short chunks over the 8-bit cache (the formulas
// are in pa_attend8.cuh), for calls that HBM bounds.
//
// Work.  All steps of 32 keys of all (sequence, row block, group of HG KV heads) stand in one line, and each CTA takes an
// equal stretch of it: no work list, no claims, and every CTA reads the same number of bytes.  A CTA that begins or
// ends within a (sequence, row block, group) leaves a partial (m, l, O) in the workspace; the one that takes its first
// step notes how many there are, and a second launch joins them.  Where no group has more than a few steps (short tables or
// windows), a CTA takes whole groups instead, and there is nothing to join.
//
// A CTA is a producer warp and MB consumer warps per KV head of the group, each with 8 NQ of the row block's rows.  The
// producer fills a ring of steps by TMA, one box per block (all HG heads) for K and for V; every 32 steps, lane l looks
// up step l's blocks and scales.  (Warps that fill rings of their own spend 700 of 2700 cycles a step on it.)
//
// A consumer works on the transposed products, 32 keys at a time, S^T = K Q^T and O^T += V^T P^T, both with mma.m16n8k16
// on f16: the keys, of which there are enough, take the products' 16 rows, and the query rows come in eights.  P^T comes
// out of S^T with keys as rows, and movmatrix turns it into the other product's operand.  (With query rows as the 16: 84 us
// on 256 sequences.  With e4m3 mma on the codes as they are, and queries in e4m3 terms: as fast there, where
// HBM bounds, but nearly twice the cycles of the conversions and f16 products.)
//
// Codes come out of shared memory in 16-byte pieces with the products' dimensions and keys permuted to fit: lane
// (g, c) of a warp takes bytes 16 c .. of the key rows perm(g) and 8 + perm(g) for S (four k-steps' words), and for P V
// bytes 16 g .. of the key rows perm(2c), perm(2c + 1), whose bytes it pairs up (prmt) and converts.  perm makes both
// free of bank conflicts under the TMA swizzle (128 bytes at D 128, 64 at D 64).
#pragma once

#include <cmath>
#include <type_traits>

#include "pa_attend8.cuh"

namespace pa {

// NQ: tiles of 8 query rows of a warp; MB: warps of a head's row block; HG: KV heads of a CTA.
template <int D, int NQ, int MB, int HG>
struct Attend8Cfg {
    static constexpr int kRows = 8 * NQ * MB;                // of a row block
    static constexpr int kConsumers = HG * MB;
    static constexpr int kCtas = attend8_ctas(NQ, MB, HG);   // per SM
    // More than 8 rows a warp: the queries' fragments lie in shared memory.  24 rows: O^T alone takes 96 registers, and whole
    // warpgroups of consumers take over registers of a producer warpgroup (of which one warp works): two CTAs of 4 + 4
    // warps are launched at 128 registers, producers keep 24 and consumers get 232 (verify 147 us; 40 and 216: 159).  At D 128
    // these kernels still spill some 300 bytes a thread (stores; 450 of loads).
    static constexpr bool kWide = NQ > 1;
    static constexpr bool kSplit = NQ == 3 && kConsumers == 4;
    static constexpr int kThreads = 32 * (kConsumers + (kSplit ? 4 : 1));
    static constexpr int kQBytes = kWide ? kConsumers * NQ * D * 16 : 0;
    static constexpr int kTileBytes = kStep8 * D * HG;       // K (or V) of a step
    static constexpr int kStagesRaw = (192 * 1024 / kCtas - kQBytes) / (2 * kTileBytes);
    static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
    // (ks scale log2(e), log2 vs, 1 / vs, -) of two blocks and each head, of 64 steps: a batch of 32 is written at once, and consumers are
    // at most kStages steps behind it
    static constexpr int kNotes = HG * 32;
    static constexpr size_t kNoteOff = (size_t)kStages * 2 * kTileBytes;
    static constexpr size_t kQOff = kNoteOff + (size_t)64 * kNotes;
    static constexpr size_t kBarOff = kQOff + kQBytes;       // full and empty [kStages]
    static constexpr size_t kSmem = kBarOff + (size_t)kStages * 16 + 1024;   // + alignment slack
    static_assert(kStages >= 2, "ring");
    static_assert((kSmem + 2048) * kCtas <= 228 * 1024, "shared memory budget");
};

// The transpose of an 8 x 8 matrix of 16-bit elements, two of a row per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The physical key row (of 8) of index n of a product.
template <int D>
__device__ __forceinline__ int perm8(int n) {
    if constexpr (D == 128) return n & 1 ? (n & 6) ^ 5 : n;
    const int c = n >> 1, r = c + 2 * (c >> 1);
    return n & 1 ? r ^ 3 : r;
}
// Byte offset of 16-byte piece ch of row r of a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t piece8(int r, int ch) {
    if constexpr (D == 128) return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4));
    return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
}

// Steps of a CTA's stretch: an equal share, but at least four (128 keys) where that leaves 64 CTAs, so that a long sequence
// has not too many parts to join; fewer where there are few steps at all and only latency counts.
__device__ __forceinline__ long long share_of(const Attend8Args &a, long long total) {
    if (a.whole) return (total + a.units - 1) / a.units;   // groups, not steps
    return max(min(4ll, (total + 63) / 64), (total + a.units - 1) / a.units);
}

// Where a warp stands in the line of steps: the sequence, row block, head group and step.
struct Place8 {
    int s, rb, h, v;
    Seq8 q;
    Steps8 st;
};

template <typename T, int D, int NQ, int MB, int HG>
__global__ void __launch_bounds__(Attend8Cfg<D, NQ, MB, HG>::kThreads, Attend8Cfg<D, NQ, MB, HG>::kCtas)
    attend8_mma_kernel(const Attend8Args a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = Attend8Cfg<D, NQ, MB, HG>;
    using H = Mma16<__half>;
    constexpr int kKS = D / 16, kMT = D / 16, kRows = C::kRows;             // k-steps of S, 16-row tiles of O^T
    constexpr int kWarps = C::kThreads / 32;
    constexpr bool kTwoTerms = NQ == 1;   // of the weights in the second product (pa_attend8.cuh has both sides)
    constexpr bool kLifted = std::is_same<T, __nv_bfloat16>::value;   // queries go in as f16, by a power of two per row
    extern __shared__ unsigned char smem_raw[];
    __shared__ long long sums[kWarps];
    __shared__ int4 begin_at;  // (sequence, -, rest low, rest high) of the first step
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv, lg = __ffs(G) - 1;  // G is a power of two
    const int groups = a.Hkv / HG;
    const uint32_t notes = ring + (uint32_t)C::kNoteOff, bars = ring + (uint32_t)C::kBarOff;
    auto full = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto empty = [&](int i) { return bars + 8u * (uint32_t)(C::kStages + i); };
    const int nb = kStep8 / a.B, lb = __ffs(a.B) - 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), C::kConsumers);
        }
        fence_mbar_init();
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    griddep_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the line: steps of a sequence, over its row blocks and head groups
    auto place_seq = [&](Place8 &p, int s, bool flag) {
        p.s = s;
        p.q = seq_of(a, s, flag);
        p.st = steps_of(a, p.q.len - p.q.n, p.q.n > 0 ? p.q.len : 0, kStep8);
    };
    auto blocks_of = [&](const Seq8 &q) { return (q.n * G + kRows - 1) / kRows; };
    // (where a.whole, a group counts as one, and one without keys too: its rows are zeros)
    auto steps_in = [&](const Place8 &p) { return (long long)blocks_of(p.q) * groups * (a.whole ? 1 : p.st.count); };
    long long total = 0, each;
    {
        const int per = (a.S + C::kThreads - 1) / C::kThreads;
        const int s0 = min(a.S, (int)threadIdx.x * per), s1 = min(a.S, s0 + per);
        long long own = 0;
        bool ok = true;
        Place8 p;
        for (int s = s0; s < s1; ++s) {
            place_seq(p, s, blockIdx.x == 0);
            ok = ok && order_ok(a, s);
            own += steps_in(p);
        }
        long long incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) sums[warp] = incl;
        ok = __syncthreads_and(ok);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            a.hdr[0] = ok;
            if (!ok) set_error(a.err, PA_DEVERR_BAD_LEN);
        }
        if (!ok) return;
        long long before = incl - own;
        for (int w = 0; w < kWarps; ++w) {
            total += sums[w];
            if (w < warp) before += sums[w];
        }
        // the thread whose sequences hold the first step looks it up
        each = share_of(a, total);
        long long u = each * blockIdx.x;
        if (u >= before && u < before + own) {
            u -= before;
            for (int s = s0; s < s1; ++s) {
                place_seq(p, s, false);
                const long long mine = steps_in(p);
                if (u < mine) {
                    begin_at = make_int4(s, 0, (int)(u & 0xffffffffll), (int)(u >> 32));
                    break;
                }
                u -= mine;
            }
        }
        __syncthreads();
    }
    const int unit = blockIdx.x;
    if (each * unit >= total) return;
    int left = (int)min(each, total - each * unit);   // steps (groups) still to take

    Place8 p;
    place_seq(p, begin_at.x, false);
    {
        const long long u = (long long)(uint32_t)begin_at.z | (long long)begin_at.w << 32;
        const int of_head = a.whole ? 1 : p.st.count;
        const long long head = u / of_head;
        p.v = (int)(u % of_head);
        p.h = (int)(head % groups);
        p.rb = (int)(head / groups);
    }
    auto next_head = [&](Place8 &p) {  // the first step of the next group (there is one)
        p.v = 0;
        if (++p.h < groups) return;
        p.h = 0;
        if (++p.rb < blocks_of(p.q)) return;
        p.rb = 0;
        do place_seq(p, p.s + 1, false);
        while (steps_in(p) == 0 && p.s + 1 < a.S);
    };
    auto first_key = [&](const Place8 &x) { return (x.v < x.st.ns ? x.v : x.v + x.st.gap) * kStep8; };

    if (warp >= C::kConsumers) {
        // ------------------------------------------------------------ producer
        if constexpr (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 24;\n" ::: "memory");
        if (warp > C::kConsumers) return;
        const uint64_t pol = policy_evict_first();
        int z[2] = {-1, -1}, issued = 0;   // per lane: the blocks of the batch's step `lane` (first head's index, or -1)
        bool ok = true;
        while (ok && left > 0) {
            const int n = a.whole ? p.st.count : min(left, p.st.count - p.v);
            for (int i = 0; ok && i < n; ++i, ++issued, ++p.v) {
                const int turn = i & 31;
                if (turn == 0) {
                    Place8 x = p;
                    x.v += lane;
                    const int key = first_key(x);
                    const bool mine = i + lane < n;
                    const int seen_from = a.window > 0 ? p.q.len - p.q.n - a.window + 1 : 0;   // by the sequence's first row
                    const uint32_t at = notes + (uint32_t)(C::kNotes * ((issued + lane) & 63));
                    int id[2];
                    bool want[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int k = key + b * a.B;
                        // only blocks that some row sees: behind a window, half a step of two blocks may be none of them
                        want[b] = b < nb && mine && k < p.q.len && (k + a.B > seen_from || k < a.sinks);
                        id[b] = want[b] ? a.block_tables[(size_t)p.s * a.max_blocks + (k >> lb)] : 0;
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const bool there = want[b] && id[b] >= 0 && id[b] < a.N;
                        if (want[b] && !there) set_error(a.err, PA_DEVERR_BAD_BLOCK);
                        z[b] = there ? id[b] * a.Hkv + p.h * HG : -1;
                    }
                    // a block that is not there has no scale; the second half of a block of 32 has the first's
                    const int from[2] = {z[0], nb == 1 ? z[0] : z[1]};
                    // as many scales on their way together as there are registers for (one head at a time: windows 56.9 us, so 55.7)
                    constexpr int kB = C::kSplit ? 1 : 2;
                    if (mine) {
#pragma unroll
                        for (int b0 = 0; b0 < 2; b0 += kB) {
                            float ks[kB][HG], vs[kB][HG];
#pragma unroll
                            for (int b = 0; b < kB; ++b)
#pragma unroll
                                for (int h = 0; h < HG; ++h) {
                                    ks[b][h] = a.k_scales[max(from[b0 + b], 0) + h];
                                    vs[b][h] = a.v_scales[max(from[b0 + b], 0) + h];
                                }
#pragma unroll
                            for (int b = 0; b < kB; ++b)
#pragma unroll
                                for (int h = 0; h < HG; ++h) {
                                    const float k1 = from[b0 + b] >= 0 ? ks[b][h] * (a.scale * kLog2e8) : 0.f, v1 = from[b0 + b] >= 0 ? vs[b][h] : -1.f;
                                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %3};" ::"r"(at + 32 * h + 16 * (b0 + b)), "f"(k1),
                                                 "f"(v1 > 0.f ? lg2(v1) : 0.f), "f"(1.f / v1)
                                                 : "memory");
                                }
                        }
                    }
                    __syncwarp();
                }
                const int st = issued % C::kStages;
                const int z0 = __shfl_sync(0xffffffffu, z[0], turn), z1 = __shfl_sync(0xffffffffu, z[1], turn);
                if (issued >= C::kStages) ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty(st), (uint32_t)((issued / C::kStages) - 1) & 1u, kWaitLimit));
                if (ok && lane == 0) {
                    const uint32_t dst = ring + (uint32_t)(st * 2 * C::kTileBytes);
                    const int there = (z0 >= 0) + (z1 >= 0);
                    if (there) mbar_arrive_expect_tx(full(st), (uint32_t)(there * 2 * a.B * D * HG));
                    else mbar_arrive(full(st));
                    if (z0 >= 0) {
                        tma_load_3d(dst, &tmk, 0, 0, z0, full(st), pol);
                        tma_load_3d(dst + C::kTileBytes, &tmv, 0, 0, z0, full(st), pol);
                    }
                    if (z1 >= 0) {
                        tma_load_3d(dst + (uint32_t)(a.B * D * HG), &tmk, 0, 0, z1, full(st), pol);
                        tma_load_3d(dst + (uint32_t)(C::kTileBytes + a.B * D * HG), &tmv, 0, 0, z1, full(st), pol);
                    }
                }
                __syncwarp();
            }
            left -= a.whole ? 1 : n;
            if (ok && left > 0) next_head(p);
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
        // the shared memory outlives its copies
        for (int k = max(0, issued - C::kStages); k < issued; ++k)
            mbar_wait_bounded(full(k % C::kStages), (uint32_t)(k / C::kStages) & 1u, kWaitLimit);
        return;
    }

    // ------------------------------------------------------------ consumers
    if constexpr (C::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n" ::: "memory");
    const int head = warp % HG, member = warp / HG;        // of the group, of the row block's warps
    const uint32_t head_at = (uint32_t)(head * a.B * D);   // of a box
    const uint32_t half_at = (uint32_t)(a.B == 16 ? 16 * D * HG : 16 * D);   // from key 0 to key 16 of a head
    bool timed_out = false;
    // the line's stretch, a (sequence, row block, group) at a time
    const int g = lane >> 2, c = lane & 3;
    int taken = 0;
    bool first_piece = true;
    while (left > 0) {
        const int n = a.whole ? p.st.count : min(left, p.st.count - p.v);   // steps of this head
        const bool whole = n == p.st.count;
        const int kvh = p.h * HG + head;
        const int r0 = p.rb * kRows + 8 * NQ * member;       // first row of the warp: row r is token r / G, head r % G
        const bool any = r0 < p.q.n * G;
        // queries as B fragments (lane (g, c): row g of a tile); what belongs to the rows 2 c, 2 c + 1 that a lane has of S^T
        uint32_t qb[kKS][C::kWide ? 1 : NQ][2];
        const uint32_t q_at = ring + (uint32_t)C::kQOff + (uint32_t)(warp * NQ * D * 16 + lane * 16);   // [k-step pair][tile][lane]: two k-steps
        float qs[NQ][2];                                     // one over the row's factor (bf16)
        int pos[NQ][2];
#pragma unroll
        for (int t8 = 0; t8 < NQ; ++t8) {
            const int tq = C::kWide ? 0 : t8;
            const int r = r0 + 8 * t8 + g;
            const bool on = r < p.q.n * G;
            const int t = on ? r >> lg : 0;
            const uint16_t *row = static_cast<const uint16_t *>(a.q) +
                                  ((size_t)(p.q.q0 + t) * a.Hq + kvh * G + (on ? r & (G - 1) : 0)) * D;
            float top = 0.f;
#pragma unroll
            for (int ch = 0; ch < D / 64; ++ch) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (on) {
                    x = *reinterpret_cast<const uint4 *>(row + 16 * (c + 4 * ch));
                    y = *reinterpret_cast<const uint4 *>(row + 16 * (c + 4 * ch) + 8);
                }
                qb[4 * ch][tq][0] = x.x, qb[4 * ch][tq][1] = x.y, qb[4 * ch + 1][tq][0] = x.z, qb[4 * ch + 1][tq][1] = x.w;
                qb[4 * ch + 2][tq][0] = y.x, qb[4 * ch + 2][tq][1] = y.y, qb[4 * ch + 3][tq][0] = y.z, qb[4 * ch + 3][tq][1] = y.w;
            }
            float back = 1.f;
            if constexpr (kLifted) {   // as f16, the row's largest at 2^10
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = Mma16<T>::unpack(qb[ks][tq][i]);
                        top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(126, 10 - ((int)(__float_as_uint(top) >> 23) - 127));   // -118 .. 126; what 2^126 lifts is exact in f16
                const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = Mma16<T>::unpack(qb[ks][tq][i]);
                        qb[ks][tq][i] = H::pack(v.x * up, v.y * up);
                    }
            }
            if constexpr (C::kWide) {
#pragma unroll
                for (int ks = 0; ks < kKS; ks += 2)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(q_at + (uint32_t)((ks / 2 * NQ + t8) * 512)), "r"(qb[ks][0][0]),
                                 "r"(qb[ks][0][1]), "r"(qb[ks + 1][0][0]), "r"(qb[ks + 1][0][1])
                                 : "memory");
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                qs[t8][o] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + o));
                const int ro = r0 + 8 * t8 + 2 * c + o;
                pos[t8][o] = ro < p.q.n * G ? p.q.len - p.q.n + (ro >> lg) : p.q.len - 1;
            }
        }
        // keys that every row of the warp sees: up to its first row's position, and above its last row's window
        const int t_first = min(p.q.n - 1, r0 >> lg), t_last = min(p.q.n - 1, (r0 + 8 * NQ - 1) >> lg);
        const int pos_first = p.q.len - p.q.n + t_first, pos_last = p.q.len - p.q.n + t_last;
        const int seen_from = a.window > 0 ? pos_first - a.window + 1 : 0;   // below: only sinks are seen by some row
        const int whole_from = a.window > 0 ? pos_last - a.window + 1 : 0;

        float o[kMT][NQ][4];    // O^T: columns (D / 8) g + 2 j + (0, 1), of the rows 2 c, 2 c + 1
        float m[NQ][2], l[NQ][2];   // m: the weights' reference (log2); l: this lane's keys only
#pragma unroll
        for (int t8 = 0; t8 < NQ; ++t8) {
#pragma unroll
            for (int j = 0; j < kMT; ++j) o[j][t8][0] = o[j][t8][1] = o[j][t8][2] = o[j][t8][3] = 0.f;
            m[t8][0] = m[t8][1] = -INFINITY, l[t8][0] = l[t8][1] = 0.f;
        }

        for (int i = 0; i < n; ++i) {
            const int st = taken % C::kStages;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(full(st), (uint32_t)(taken / C::kStages) & 1u, kWaitLimit))) timed_out = true;
            if (timed_out) break;
            if (any) {
                const int kb = first_key(p);
                const uint32_t kst = ring + (uint32_t)(st * 2 * C::kTileBytes) + head_at, vst = kst + C::kTileBytes;
                float ks[2], lv[2], iv[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float pad;
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(ks[b]), "=f"(lv[b]), "=f"(iv[b]), "=f"(pad)
                                 : "r"(notes + (uint32_t)(C::kNotes * (taken & 63) + 32 * head + 16 * b)));
                }
                const bool clear = kb + kStep8 - 1 <= pos_first && (kb >= whole_from || kb + kStep8 <= a.sinks) && iv[0] > 0.f && iv[1] > 0.f;
                // Both halves of the step go through each stage together; where registers are short (more rows a warp, or
                // twelve warps) one after the other.
                constexpr int kKK = NQ == 1 && C::kConsumers <= 8 ? 2 : 1;
#pragma unroll 1
                for (int k0 = 0; k0 < 2; k0 += kKK) {
                    // the notes of half i2 of this turn
                    auto of_half = [&](const float (&x)[2], int i2) { return kKK == 2 ? x[i2] : k0 ? x[1] : x[0]; };
                    // ---- S^T = K Q^T, 16 keys at a time: rows g (key perm(g)) and g + 8, columns 2 c, 2 c + 1 of each tile
                    float s[kKK][NQ][4];
#pragma unroll
                    for (int i2 = 0; i2 < kKK; ++i2)
#pragma unroll
                        for (int t8 = 0; t8 < NQ; ++t8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[i2][t8][e] = 0.f;
#pragma unroll
                    for (int ch = 0; ch < D / 64; ++ch) {
                        uint4 lo[kKK], hi[kKK];
#pragma unroll
                        for (int i2 = 0; i2 < kKK; ++i2) {
                            const uint32_t at = kst + (k0 + i2 ? half_at : 0u);
                            lo[i2] = lds128(at + piece8<D>(perm8<D>(g), c + 4 * ch));
                            hi[i2] = lds128(at + piece8<D>(8 + perm8<D>(g), c + 4 * ch));
                        }
#pragma unroll
                        for (int w2 = 0; w2 < 4; w2 += 2) {
                            uint4 q4[C::kWide ? NQ : 1];
                            if constexpr (C::kWide) {
#pragma unroll
                                for (int t8 = 0; t8 < NQ; ++t8) q4[t8] = lds128(q_at + (uint32_t)(((2 * ch + w2 / 2) * NQ + t8) * 512));
                            }
#pragma unroll
                            for (int w = w2; w < w2 + 2; ++w)
#pragma unroll
                                for (int i2 = 0; i2 < kKK; ++i2) {
                                    const uint32_t x = w == 0 ? lo[i2].x : w == 1 ? lo[i2].y : w == 2 ? lo[i2].z : lo[i2].w;
                                    const uint32_t y = w == 0 ? hi[i2].x : w == 1 ? hi[i2].y : w == 2 ? hi[i2].z : hi[i2].w;
                                    const uint32_t a0 = f16_of_codes(x & 0xffffu), a1 = f16_of_codes(y & 0xffffu);
                                    const uint32_t a2 = f16_of_codes(x >> 16), a3 = f16_of_codes(y >> 16);
#pragma unroll
                                    for (int t8 = 0; t8 < NQ; ++t8) {
                                        if constexpr (C::kWide) H::mma(s[i2][t8], a0, a1, a2, a3, w & 1 ? q4[t8].z : q4[t8].x, w & 1 ? q4[t8].w : q4[t8].y);
                                        else H::mma(s[i2][t8], a0, a1, a2, a3, qb[4 * ch + w][t8][0], qb[4 * ch + w][t8][1]);
                                    }
                                }
                        }
                    }
#pragma unroll
                    for (int i2 = 0; i2 < kKK; ++i2) {
                        const int kk = k0 + i2;
                        // a_j = z_j + log2 vs
#pragma unroll
                        for (int t8 = 0; t8 < NQ; ++t8) {
                            // (a row's factor, of up to 2^126, meets the scales only here: either may be far from 1 alone)
                            const float ck = of_half(ks, i2);
                            const float mul[2] = {kLifted ? qs[t8][0] * ck : ck, kLifted ? qs[t8][1] * ck : ck};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float x = fmaf(s[i2][t8][e], mul[e & 1], of_half(lv, i2));
                                if (!clear) {
                                    const int j = kb + 16 * kk + 8 * (e >> 1) + perm8<D>(g);
                                    if (!(of_half(iv, i2) > 0.f && j <= pos[t8][e & 1] && (a.window == 0 || j > pos[t8][e & 1] - a.window || j < a.sinks)))
                                        x = -INFINITY;
                                }
                                s[i2][t8][e] = x;
                            }
                        }
                    }
                    // this lane's bytes of its four keys' rows of V
                    uint32_t vw[kKK][4][D / 32];
                    auto load_v = [&](int i2) {
                        const int kk = k0 + i2;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int row = 8 * (e >> 1) + perm8<D>(2 * c + (e & 1));
                            const uint32_t tile = vst + (kk ? half_at : 0u);
                            if constexpr (D == 128) {
                                const uint4 x = lds128(tile + piece8<D>(row, g));
                                vw[i2][e][0] = x.x, vw[i2][e][1] = x.y, vw[i2][e][2] = x.z, vw[i2][e][3] = x.w;
                            } else {
                                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                             : "=r"(vw[i2][e][0]), "=r"(vw[i2][e][1])
                                             : "r"(tile + piece8<D>(row, g >> 1) + 8 * (g & 1)));
                            }
                            if (!clear) {  // a key that no row sees may hold anything
                                const int j = kb + 16 * kk + row;
                                if (!(of_half(iv, i2) > 0.f && j <= pos_last && (j >= seen_from || j < a.sinks))) {
#pragma unroll
                                    for (int x = 0; x < D / 32; ++x) vw[i2][e][x] = 0u;
                                }
                            }
                        }
                    };
                    if constexpr (NQ < 3) load_v(0);   // (24 rows a warp: registers for it come free later)
                    // ---- the running reference
                    bool need = false;
                    float mx[NQ][2];
#pragma unroll
                    for (int t8 = 0; t8 < NQ; ++t8)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            mx[t8][e] = fmaxf(s[0][t8][e], s[0][t8][2 + e]);
                            if constexpr (kKK == 2) mx[t8][e] = fmaxf(mx[t8][e], fmaxf(s[1][t8][e], s[1][t8][2 + e]));
                            need = need || mx[t8][e] > m[t8][e] + (8.f + kLift8);
                        }
                    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                        for (int t8 = 0; t8 < NQ; ++t8)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x = mx[t8][e];
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                                x = fmaxf(m[t8][e], x - kLift8);
                                const float alpha = x == -INFINITY ? 1.f : ex2(m[t8][e] - x);
                                m[t8][e] = x;
                                l[t8][e] *= alpha;
#pragma unroll
                                for (int j = 0; j < kMT; ++j) {
                                    o[j][t8][e] *= alpha;
                                    o[j][t8][2 + e] *= alpha;
                                }
                            }
                    }
                    // ---- weights, as B fragments: keys as k
                    uint32_t pb[kKK][NQ][2], pl[kKK][kTwoTerms ? NQ : 1][2];
#pragma unroll
                    for (int t8 = 0; t8 < NQ; ++t8) {
                        const float m0 = m[t8][0] == -INFINITY ? 0.f : m[t8][0], m1 = m[t8][1] == -INFINITY ? 0.f : m[t8][1];
#pragma unroll
                        for (int i2 = 0; i2 < kKK; ++i2) {
                            const float w0 = ex2(s[i2][t8][0] - m0), w1 = ex2(s[i2][t8][1] - m1), w2 = ex2(s[i2][t8][2] - m0), w3 = ex2(s[i2][t8][3] - m1);
                            // a block that is not there has weights of 0 (and an iv of -1)
                            l[t8][0] = fmaf(w0 + w2, of_half(iv, i2), l[t8][0]);
                            l[t8][1] = fmaf(w1 + w3, of_half(iv, i2), l[t8][1]);
                            const uint32_t h0 = H::pack(w0, w1), h1 = H::pack(w2, w3);
                            pb[i2][t8][0] = transpose8(h0);
                            pb[i2][t8][1] = transpose8(h1);
                            if constexpr (kTwoTerms) {   // what the rounding left
                                const float2 f0 = H::unpack(h0), f1 = H::unpack(h1);
                                pl[i2][t8][0] = transpose8(H::pack(w0 - f0.x, w1 - f0.y));
                                pl[i2][t8][1] = transpose8(H::pack(w2 - f1.x, w3 - f1.y));
                            }
                        }
                    }
                    // ---- O^T += V^T P^T
                    if constexpr (NQ >= 3) load_v(0);
                    if constexpr (kKK == 2) load_v(1);
#pragma unroll
                    for (int i2 = 0; i2 < kKK; ++i2)
#pragma unroll
                        for (int j = 0; j < kMT; ++j) {
                            const int x = j >> 1;
                            const uint32_t lo = __byte_perm(vw[i2][0][x], vw[i2][1][x], j & 1 ? 0x7362 : 0x5140);
                            const uint32_t hi = __byte_perm(vw[i2][2][x], vw[i2][3][x], j & 1 ? 0x7362 : 0x5140);
                            const uint32_t a0 = f16_of_codes(lo & 0xffffu), a1 = f16_of_codes(lo >> 16);
                            const uint32_t a2 = f16_of_codes(hi & 0xffffu), a3 = f16_of_codes(hi >> 16);
#pragma unroll
                            for (int t8 = 0; t8 < NQ; ++t8) {
                                H::mma(o[j][t8], a0, a1, a2, a3, pb[i2][t8][0], pb[i2][t8][1]);
                                if constexpr (kTwoTerms) H::mma(o[j][t8], a0, a1, a2, a3, pl[i2][t8][0], pl[i2][t8][1]);
                            }
                        }
                }
            }
            __syncwarp();  // every lane has read the stage
            if (lane == 0) mbar_arrive(empty(st));
            ++taken;
            ++p.v;
        }
        left -= a.whole ? 1 : n;
        if (timed_out) {
            if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
            break;
        }

        // ---- the outputs, or this CTA's part of them
        const int slot = first_piece ? 2 * unit : 2 * unit + 1;
        float *part = a.parts + ((size_t)slot * HG + head) * kRows * (D + 2);
        if (p.v == n && warp == 0 && lane == 0) {
            // it took the group's first step: the rest is the following CTAs'
            int2 *note = reinterpret_cast<int2 *>(a.list) + ((size_t)p.s * groups + p.h) * ((a.max_query_len * G + kRows - 1) / kRows) + p.rb;
            *note = make_int2(slot, whole ? 0 : 1 + (int)((p.st.count - n + each - 1) / each));
        }
#pragma unroll
        for (int t8 = 0; t8 < NQ; ++t8)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[t8][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = 8 * NQ * member + 8 * t8 + 2 * c + e, r = p.rb * kRows + row;
                if (r >= p.q.n * G) continue;
                const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                float v[D / 8];
#pragma unroll
                for (int j = 0; j < kMT; ++j) v[2 * j] = o[j][t8][e] * inv, v[2 * j + 1] = o[j][t8][2 + e] * inv;
                if (!whole) {
                    float4 *to = reinterpret_cast<float4 *>(part + (size_t)row * D + D / 8 * g);
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) to[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                    if (g == 0) *reinterpret_cast<float2 *>(part + (size_t)kRows * D + 2 * row) = make_float2(m[t8][e], sum);
                    continue;
                }
                const size_t at = ((size_t)(p.q.q0 + (r >> lg)) * a.Hq + kvh * G + (r & (G - 1))) * D + D / 8 * g;
                if (a.out16) {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        to[x] = make_uint4(Mma16<T>::pack(v[8 * x], v[8 * x + 1]), Mma16<T>::pack(v[8 * x + 2], v[8 * x + 3]),
                                           Mma16<T>::pack(v[8 * x + 4], v[8 * x + 5]), Mma16<T>::pack(v[8 * x + 6], v[8 * x + 7]));
                } else {
                    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) to[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                }
            }
        first_piece = false;
        if (left > 0) next_head(p);
    }
}

// CTA x takes (sequence, KV head, row block) x, and of its kRows rows every gridDim.y-th from y on: it joins their parts,
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,   M = max m_i,
// and writes the zeros of a sequence without keys.  No more parts than warps: a warp takes a row, a lane D / 32 of its
// columns.  More: the warps share out a row's parts, and what they make of them is joined once more.  (One sequence of
// 32768 keys, 146 parts a head: the call 52.6 us with a warp a row, 33.3 so.  256 sequences, 2048 joins of 4 rows: 80.0 us
// with 4 warps, 82.2 with 8.)
constexpr int kMergeWarps8 = 8;
// Parts i0, i0 + step .. of n (the first one apart, the others by `stride`) joined for kN rows from `row` on, `apart` from each
// other: a lane's columns relative to the rows' largest m.
template <int kN, int D>
__device__ __forceinline__ void join8(const float *first, const float *later, size_t stride, int n, int kRows, int row, int apart, int i0, int step,
                                      int lane, float (&M)[kN], float (&l)[kN], float (&o)[kN][D / 32]) {
    constexpr int kPer = D / 32;
#pragma unroll
    for (int r = 0; r < kN; ++r) M[r] = -INFINITY;
    for (int i = i0 + step * lane; i < n; i += 32 * step) {
        const float *at = (i == 0 ? first : later + (size_t)(i - 1) * stride) + (size_t)kRows * D + 2 * row;
#pragma unroll
        for (int r = 0; r < kN; ++r) M[r] = fmaxf(M[r], at[2 * r * apart]);
    }
#pragma unroll
    for (int r = 0; r < kN; ++r) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M[r] = fmaxf(M[r], __shfl_xor_sync(0xffffffffu, M[r], x));
        l[r] = 0.f;
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[r][x] = 0.f;
    }
#pragma unroll 4
    for (int i = i0; i < n; i += step) {
        const float *at = i == 0 ? first : later + (size_t)(i - 1) * stride;
#pragma unroll
        for (int r = 0; r < kN; ++r) {
            const int mine = row + r * apart;
            const float2 ml = *reinterpret_cast<const float2 *>(at + (size_t)kRows * D + 2 * mine);
            const float w = ex2(ml.x - (M[r] == -INFINITY ? 0.f : M[r]));
            l[r] = fmaf(w, ml.y, l[r]);
#pragma unroll
            for (int x = 0; x < kPer; x += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(at + (size_t)mine * D + kPer * lane + x);
                o[r][x] = fmaf(w, v.x, o[r][x]);
                o[r][x + 1] = fmaf(w, v.y, o[r][x + 1]);
            }
        }
    }
}
template <typename T, int D, int HG>
__global__ void __launch_bounds__(32 * kMergeWarps8) attend8_merge_kernel(const Attend8Args a, int kRows, int nrb) {
    constexpr int kPer = D / 32;
    __shared__ float some[kMergeWarps8][D], some_m[kMergeWarps8], some_l[kMergeWarps8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    griddep_wait();
    const int G = a.Hq / a.Hkv;
    const int s = blockIdx.x / (a.Hkv * nrb), h = blockIdx.x / nrb % a.Hkv, rb = blockIdx.x % nrb;
    if (!a.hdr[0]) return;
    const Seq8 q = seq_of(a, s, false);
    if (rb * kRows >= q.n * G) return;
    int2 note = make_int2(0, 0);   // the first part's slot, and how many there are
    if (q.len > 0) {
        note = reinterpret_cast<const int2 *>(a.list)[((size_t)s * (a.Hkv / HG) + h / HG) * nrb + rb];
        if (note.y == 0) return;
        // (the note of a group whose first step timed out was not written: the parts that are read exist all the same)
        if (note.y < 0 || note.x < 0 || note.x >= 2 * a.units || note.y > a.units - note.x / 2) return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    // the parts: the first in slot note.x, the others in the following CTAs' first slots
    auto part = [&](int i) { return a.parts + ((size_t)(i == 0 ? note.x : 2 * (note.x / 2 + i)) * HG + h % HG) * kRows * (D + 2); };
    const float *first = part(0), *later = part(1);
    const size_t stride = (size_t)2 * HG * kRows * (D + 2);
    auto write = [&](int row, float l, const float (&o)[kPer]) {
        const int r = rb * kRows + row, t = r / G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = ((size_t)(q.q0 + t) * a.Hq + h * G + (r - t * G)) * D + kPer * lane;
        if (a.out16) {
            uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at);
#pragma unroll
            for (int x = 0; x < kPer / 2; ++x) to[x] = Mma16<T>::pack(o[2 * x] * inv, o[2 * x + 1] * inv);
        } else {
#pragma unroll
            for (int x = 0; x < kPer; ++x) static_cast<float *>(a.out)[at + x] = o[x] * inv;
        }
    };
    const int rows = min(kRows, q.n * G - rb * kRows);
    float M[1], l[1], o[1][kPer];
    if (note.y <= warps) {
        const int apart = gridDim.y * warps;
        int row = blockIdx.y + gridDim.y * warp;
        for (; row + apart < rows; row += 2 * apart) {   // two rows' loads under way: five drafted tokens 149.7 -> 145.7 us (four: 149.1)
            float M2[2], l2[2], o2[2][kPer];
            join8<2, D>(first, later, stride, note.y, kRows, row, apart, 0, 1, lane, M2, l2, o2);
            write(row, l2[0], o2[0]);
            write(row + apart, l2[1], o2[1]);
        }
        if (row < rows) {
            join8<1, D>(first, later, stride, note.y, kRows, row, 0, 0, 1, lane, M, l, o);
            write(row, l[0], o[0]);
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        join8<1, D>(first, later, stride, note.y, kRows, row, 0, warp, warps, lane, M, l, o);
#pragma unroll
        for (int x = 0; x < kPer; ++x) some[warp][kPer * lane + x] = o[0][x];
        if (lane == 0) some_m[warp] = M[0], some_l[warp] = l[0];
        __syncthreads();
        if (warp == 0) {
            float top = -INFINITY;
            for (int w = 0; w < warps; ++w) top = fmaxf(top, some_m[w]);
            if (top == -INFINITY) top = 0.f;
            l[0] = 0.f;
#pragma unroll
            for (int x = 0; x < kPer; ++x) o[0][x] = 0.f;
            for (int w = 0; w < warps; ++w) {
                const float by = ex2(some_m[w] - top);
                l[0] = fmaf(by, some_l[w], l[0]);
#pragma unroll
                for (int x = 0; x < kPer; ++x) o[0][x] = fmaf(by, some[w][kPer * lane + x], o[0][x]);
            }
            write(row, l[0], o[0]);
        }
        __syncthreads();
    }
}

template <typename T, int D, int NQ, int MB, int HG>
cudaError_t launch_attend8_t(const Attend8Args &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    using C = Attend8Cfg<D, NQ, MB, HG>;
    static std::atomic<int> configured[kMaxLaunchDevices];
    int one = 0;
    cudaError_t e = per_device_value(configured, &one, [](int, int *v) {
        *v = 1;
        return cudaFuncSetAttribute(attend8_mma_kernel<T, D, NQ, MB, HG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.units);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend8_mma_kernel<T, D, NQ, MB, HG>, a, tmk, tmv);
    if (e != cudaSuccess || a.whole) return e;
    // the join: a CTA per (sequence, KV head, row block)
    const long long blocks = ((long long)a.max_query_len * (a.Hq / a.Hkv) + C::kRows - 1) / C::kRows;
    if (blocks * a.S * a.Hkv > 0x7fffffffLL) return cudaErrorInvalidValue;
    const long long joins = blocks * a.S * a.Hkv;
    // few of them: their rows in CTAs of their own
    const long long split = (4 * kSms8 + joins - 1) / joins;
    cfg.gridDim = dim3((unsigned)joins, (unsigned)(split < C::kRows ? split : C::kRows));
    cfg.blockDim = dim3(split > 1 ? 32 * kMergeWarps8 : 128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attend8_merge_kernel<T, D, HG>, a, (int)C::kRows, (int)blocks);
}

template <typename T, int D, int NQ, int MB>
cudaError_t dispatch_heads(const Attend8Args &a, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    if constexpr (NQ * MB < 6)
        if (hg == 4) return launch_attend8_t<T, D, NQ, MB, 4>(a, tmk, tmv, st);
    return hg == 2 ? launch_attend8_t<T, D, NQ, MB, 2>(a, tmk, tmv, st) : launch_attend8_t<T, D, NQ, MB, 1>(a, tmk, tmv, st);
}
template <typename T, int D>
cudaError_t dispatch_attend8(const Attend8Args &a, Rows8 r, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    if (r.nq == 1) return r.mb == 1 ? dispatch_heads<T, D, 1, 1>(a, hg, tmk, tmv, st) : dispatch_heads<T, D, 1, 2>(a, hg, tmk, tmv, st);
    if (r.nq == 3) return r.mb == 1 ? dispatch_heads<T, D, 3, 1>(a, hg, tmk, tmv, st) : dispatch_heads<T, D, 3, 2>(a, hg, tmk, tmv, st);
    return r.mb == 2 ? dispatch_heads<T, D, 2, 2>(a, hg, tmk, tmv, st) : dispatch_heads<T, D, 2, 4>(a, hg, tmk, tmv, st);
}

}  // namespace pa
