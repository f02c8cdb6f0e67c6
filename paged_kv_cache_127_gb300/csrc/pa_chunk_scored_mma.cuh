// pa_chunk_scored_mma.cuh -- scored chunk attention for short query chunks
// (drafted tokens being verified) on mma.m16n8k16.
//
// For the query row at position pos and the keys j of its own range [begin, end)
//   z_j = cap(scale q.k_j) - slope_h |pos - j|,   out = sum_j softmax(z)_j v_j.
// The structure and tile configuration are those of the plain short-chunk kernel
// (pa_chunk_mma.cuh): an item is (sequence, context partition, group of HG KV
// heads, row block), HG x RW consumer warps hold 16-row tiles of (query token,
// query head) rows, one producer warp streams 16-key chunks by TMA, and the
// eight-warp CTA splits its registers so that a consumer takes two chunks a step.
//
// What differs: an item holds the keys [lo, hi) of its partition that some of its
// rows see and streams from the chunk of lo; each row masks to its own range; a
// warp skips chunks that none of its rows sees; cap and bias are applied to the
// logits; V rows that no row of a warp sees are zeroed in its B fragments.
//
// Finish: a row whose range lies in one partition writes out[]; otherwise its
// partitions store (m, l, acc) and the merge combines those the range touches.
//
// Bound: HBM (a chunk's rows share each key).
// Measured: five drafted tokens of 256 sequences (32 / 8 heads, D 128, bf16, capped) 133 us (floor 116), 128 of them
// this kernel's.
#pragma once

#include <cuda.h>

#include <climits>
#include <cmath>

#include "pa_chunk_mma.cuh"
#include "pa_score.cuh"

namespace pa {

// Zeroes the V rows of a 16-key chunk whose bit of `any` is not set, in a lane's B fragments (words 0 and 2 hold
// keys c2, c2 + 1; 1 and 3 keys c2 + 8, c2 + 9): a weight of 0 does not keep out what may be NaN.
template <int N>
__device__ __forceinline__ void keep_seen(uint32_t (&bv)[N][4], uint32_t any, int c2) {
    const uint32_t lo = any >> c2, hi = any >> (c2 + 8);
    const uint32_t mlo = (lo & 1u ? 0x0000ffffu : 0u) | (lo & 2u ? 0xffff0000u : 0u);
    const uint32_t mhi = (hi & 1u ? 0x0000ffffu : 0u) | (hi & 2u ? 0xffff0000u : 0u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        bv[i][0] &= mlo;
        bv[i][1] &= mhi;
        bv[i][2] &= mlo;
        bv[i][3] &= mhi;
    }
}

template <typename T, int D, int HG, int RW>
__global__ void __launch_bounds__(ChunkCfg<D, HG, RW>::kThreads, ChunkCfg<D, HG, RW>::kMinBlocks)
    scored_chunk_kernel(const ScoredArgs a, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv) {
    using C = ChunkCfg<D, HG, RW>;
    using M = Mma16<T>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // 1024-aligned: the 128-byte swizzle repeats every 1 KB
    unsigned char *basep = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv;
    const int Pt = a.partition_size;
    const int ngroups = a.Hkv / HG;
    const int lb = __ffs(a.B) - 1;  // block_size is a power of two

    const uint32_t full0 = base + (uint32_t)C::kFullOff;
    const uint32_t empty0 = base + (uint32_t)C::kEmptyOff;
    const uint32_t ifull0 = base + (uint32_t)C::kItemFullOff;
    const uint32_t iempty0 = base + (uint32_t)C::kItemEmptyOff;
    // [slot * 3]: (s, p, lo, hi), (g0, chunks, valid, query_start[s]), (n_s, len_s, row block, -)
    int4 *info = reinterpret_cast<int4 *>(basep + C::kInfoOff);
    int32_t *tbl = reinterpret_cast<int32_t *>(basep + C::kTblOff);  // [slot][kTblCap]

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, C::kConsumers);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(ifull0 + 8 * i, 1);
            mbar_init(iempty0 + 8 * i, C::kConsumers);
        }
        fence_mbar_init();
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    __syncthreads();
    griddep_wait();  // the plan kernel's work list must be complete
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int n_items = a.plan_hdr[0] > 0 ? a.plan_hdr[0] * ngroups : 0;

    // ---- lane roles in the MMA fragments
    const int g = lane >> 2;         // fragment rows g and g + 8
    const int c2 = (lane & 3) * 2;   // fragment column pair
    const int lm = lane >> 3;        // ldmatrix: which 8x8 matrix this lane addresses
    const int lr = lane & 7;         // ldmatrix: which row of it
    const uint32_t kx = (uint32_t)(lm ^ lr);          // swizzled chunk bits for K reads
    const uint32_t vx = (uint32_t)((lm >> 1) ^ lr);   // and for V reads
    const ScoreCap score(a);
    const float sl = a.scale * kLog2e;
    const CapFit fit(score.in);
    // dot products to logits in log2 units
    auto to_log2 = [&](auto &f) {
        constexpr int N = sizeof(f) / sizeof(f[0]);
        if (score.cap && sl > 0.f) {
            float most = fabsf(f[0]);
#pragma unroll
            for (int i = 1; i < N; ++i) most = fmaxf(most, fabsf(f[i]));
            cap_in_place(f, fit, most);
        }
        if (score.cap && !(sl > 0.f)) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = score(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] *= sl;
        }
    };
    const int head = warp % HG;      // KV head of the item's group
    const int tile_of = warp / HG;   // row tile within the item's row block

    // ------------------------------------------------------------ producer warp
    // The last warp claims items, fills the item slots and issues the TMA loads,
    // up to kStages chunks ahead of the consumer warps and across item
    // boundaries; it never consumes, so a claim overlaps the chunks already in
    // the ring instead of stalling it.  First item: list entry blockIdx.x; later
    // ones are claimed from the counter when the issue cursor reaches them, not
    // earlier, so each CTA's last item is taken as late as possible and the
    // largest-first order bounds the tail.
    if (warp >= C::kConsumers) {
        if constexpr (C::kRegSplit) {
            // launched at 168 registers a thread (3 warps per scheduler): the
            // producer warpgroup gives up all but 40, the two consumer warpgroups
            // take 232 (8 x 232 + 4 x 40 = 12 x 168); one warp of the group produces
            asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n" ::: "memory");
            if (warp > C::kConsumers) return;
        }
        const uint64_t pol = policy_evict_first();
        int iss = 0;  // chunks issued
        bool ok = true;
        for (int seq = 0; ok; ++seq) {
            const int slot = seq % C::kSlots;
            // every consumer warp must be done with the item that used this slot
            if (seq >= C::kSlots &&
                !mbar_wait_bounded(iempty0 + 8 * slot, (uint32_t)((seq / C::kSlots) - 1) & 1u, kWaitLimit)) {
                if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                break;
            }
            int idx = 0;
            if (lane == 0) idx = seq == 0 ? (int)blockIdx.x : (int)gridDim.x + atomicAdd(a.plan_hdr + 1, 1);
            idx = __shfl_sync(0xffffffffu, idx, 0);
            int4 e0 = make_int4(0, 0, 0, 0), e1 = make_int4(0, 0, 0, 0), e2 = make_int4(0, 0, 0, 0);
            int32_t *tb = tbl + slot * C::kTblCap;
            if (idx < n_items) {
                int4 e = a.plan_list[idx / ngroups];  // (sequence, partition | row block << 16, lo, hi)
                const int rb = e.y >> 16;
                e.y &= 0xffff;
                e0 = e;
                const int qs = a.query_start[e.x];
                const int n = a.query_start[e.x + 1] - qs;
                const int k16 = e.z & ~15;
                e1 = make_int4((idx % ngroups) * HG, (e.w - k16 + 15) >> 4, 1, qs);
                e2 = make_int4(n, a.context_lens[e.x], rb, 0);
                const int blk0 = k16 >> lb;
                const int nblk = ((e.w - 1) >> lb) - blk0 + 1;
                const int32_t *row = a.block_tables + (size_t)e.x * a.max_blocks + blk0;
                for (int i = lane; i < nblk; i += 32) {
                    int pb = row[i];
                    if (pb < 0 || pb >= a.N) {
                        set_error(a.err, PA_DEVERR_BAD_BLOCK);
                        pb = -1;
                    }
                    tb[i] = pb;
                }
            }
            if (lane == 0) {
                info[3 * slot] = e0;
                info[3 * slot + 1] = e1;
                info[3 * slot + 2] = e2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ifull0 + 8 * slot);  // release: info and table visible
            if (idx >= n_items) break;
            for (int c = 0; c < e1.y; ++c) {
                const int st = iss % C::kStages;
                // every consumer warp has released this stage's previous chunk
                if (iss >= C::kStages &&
                    !mbar_wait_bounded(empty0 + 8 * st, (uint32_t)((iss / C::kStages) - 1) & 1u, kWaitLimit)) {
                    if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t bar = full0 + 8 * st;
                    const int key = (e0.z & ~15) + 16 * c;
                    const int pb = tb[(key >> lb) - (e0.z >> lb)];
                    if (pb < 0) {
                        mbar_arrive(bar);  // bad table entry: complete the phase without data
                    } else {
                        const uint32_t dst = base + (uint32_t)(st * C::kStageBytes);
                        const int y = key & (a.B - 1);
                        const int z = pb * a.Hkv + e1.x;
                        mbar_arrive_expect_tx(bar, C::kStageBytes);
#pragma unroll
                        for (int sb = 0; sb < C::kSub; ++sb) {
                            tma_load_3d(dst + sb * C::kBoxBytes, &tmk, sb * 64, y, z, bar, pol);
                            tma_load_3d(dst + C::kTileBytes + sb * C::kBoxBytes, &tmv, sb * 64, y, z, bar, pol);
                        }
                    }
                }
                ++iss;
            }
        }
        // The CTA's shared memory outlives its copies: wait for the last
        // kStages chunks issued (one pending phase per stage at most, so the
        // parities are unambiguous); they have normally landed long ago.
        for (int k = iss > C::kStages ? iss - C::kStages : 0; k < iss; ++k)
            mbar_wait_bounded(full0 + 8 * (k % C::kStages), (uint32_t)(k / C::kStages) & 1u, kWaitLimit);
        return;
    }

    // ------------------------------------------------------------ consumer warps
    // Every consumer warp walks the same items (slot by slot) and chunks
    // (stage by stage).
    if constexpr (C::kRegSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n" ::: "memory");
    uint32_t qa[C::kKS][4];
    int cons = 0;  // chunks consumed by this warp
    for (int seq = 0;; ++seq) {
        const int slot = seq % C::kSlots;
        if (!mbar_wait_bounded(ifull0 + 8 * slot, (uint32_t)(seq / C::kSlots) & 1u, kWaitLimit)) {
            if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
            break;
        }
        const int4 e0 = info[3 * slot];
        const int4 e1 = info[3 * slot + 1];
        const int4 e2 = info[3 * slot + 2];
        if (!e1.z) break;  // no more work
        const int p = e0.y, lo = e0.z, hi = e0.w, k16 = lo & ~15, blk0 = k16 >> lb;
        const int kvh = e1.x + head;
        const int nchunk = e1.y;
        const int qs = e1.w;
        const int n = e2.x, len = e2.y;
        const int32_t *ctb = tbl + slot * C::kTblCap;

        // this lane's two query rows
        const int r0 = (e2.z * RW + tile_of) * 16 + g;
        const int r1 = r0 + 8;
        const int t0 = r0 / G, t1 = r1 / G;
        const bool v0 = t0 < n, v1 = t1 < n;
        const int h0 = kvh * G + r0 % G, h1 = kvh * G + r1 % G;
        const int pos0 = len - n + t0, pos1 = len - n + t1;
        const int2 k0 = v0 ? row_range(a, qs + t0, pos0, len) : make_int2(0, 0);  // this lane's rows' keys
        const int2 k1 = v1 ? row_range(a, qs + t1, pos1, len) : make_int2(0, 0);
        // keys that some row of this warp sees
        const int wend = __reduce_max_sync(0xffffffffu, max(k0.y, k1.y));
        const int wbegin = __reduce_min_sync(0xffffffffu, min(k0.x < k0.y ? k0.x : INT_MAX, k1.x < k1.y ? k1.x : INT_MAX));
        // keys that every row of this warp sees, among the rows that see any
        const int win0 = __reduce_max_sync(0xffffffffu, max(k0.x < k0.y ? k0.x : 0, k1.x < k1.y ? k1.x : 0));
        const int win1 = __reduce_min_sync(0xffffffffu, min(k0.x < k0.y ? k0.y : INT_MAX, k1.x < k1.y ? k1.y : INT_MAX));
        const float s0 = a.slopes ? a.slopes[h0] * kLog2e : 0.f, s1 = a.slopes ? a.slopes[h1] * kLog2e : 0.f;
        {
            const uint16_t *qb = static_cast<const uint16_t *>(a.q);
            const uint16_t *q0 = qb + ((size_t)(qs + (v0 ? t0 : 0)) * a.Hq + h0) * D;
            const uint16_t *q1 = qb + ((size_t)(qs + (v1 ? t1 : 0)) * a.Hq + h1) * D;
#pragma unroll
            for (int ks = 0; ks < C::kKS; ++ks) {
                qa[ks][0] = v0 ? *reinterpret_cast<const uint32_t *>(q0 + ks * 16 + c2) : 0u;
                qa[ks][1] = v1 ? *reinterpret_cast<const uint32_t *>(q1 + ks * 16 + c2) : 0u;
                qa[ks][2] = v0 ? *reinterpret_cast<const uint32_t *>(q0 + ks * 16 + 8 + c2) : 0u;
                qa[ks][3] = v1 ? *reinterpret_cast<const uint32_t *>(q1 + ks * 16 + 8 + c2) : 0u;
            }
        }
        float o[C::kNT][4];
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        bool timed_out = false;

        for (int j = 0; j < nchunk; ++j) {
            const int st = cons % C::kStages;
            const uint32_t parity = (uint32_t)(cons / C::kStages) & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(full0 + 8 * st, parity, kWaitLimit))) {
                if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                timed_out = true;
                break;
            }
            const int kb = k16 + 16 * j;
            const int n0 = max(lo - kb, 0);  // keys n0 .. n1 - 1 of the chunk are in the item's span
            const int n1 = ctb[(kb >> lb) - blk0] < 0 ? 0 : min(16, hi - kb);
            // two full chunks that every row of this warp sees whole (those that see anything; the others' results are
            // dropped): one softmax step over 32 keys
            const bool pair = C::kRegSplit && j + 1 < nchunk && n0 == 0 && n1 == 16 && ctb[((kb + 16) >> lb) - blk0] >= 0 &&
                              hi - kb >= 32 && kb >= win0 && kb + 32 <= min(win1, wend);
            if (pair) {
                const int st2 = (cons + 1) % C::kStages;
                const uint32_t parity2 = (uint32_t)((cons + 1) / C::kStages) & 1u;
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(full0 + 8 * st2, parity2, kWaitLimit))) {
                    if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                    timed_out = true;
                    break;
                }
                const uint32_t kstp[2] = {base + (uint32_t)(st * C::kStageBytes) + (uint32_t)(head * C::kHeadSub),
                                          base + (uint32_t)(st2 * C::kStageBytes) + (uint32_t)(head * C::kHeadSub)};
                uint32_t bv[C::kNT / 2][4];
#pragma unroll
                for (int ntp = 0; ntp < C::kNT / 2; ++ntp) {
                    const uint32_t addr = kstp[0] + C::kTileBytes + (uint32_t)((ntp >> 2) * C::kBoxBytes) +
                                          (uint32_t)(((lm & 1) * 8 + lr) * 128) +
                                          (((uint32_t)(2 * (ntp & 3)) ^ vx) << 4);
                    ldsm_x4_t(addr, bv[ntp][0], bv[ntp][1], bv[ntp][2], bv[ntp][3]);
                }
                float sc[2][2][2][4];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
                            sc[c][nt][hh][0] = sc[c][nt][hh][1] = sc[c][nt][hh][2] = sc[c][nt][hh][3] = 0.f;
#pragma unroll
                for (int ks2 = 0; ks2 < C::kKS / 2; ++ks2) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const uint32_t addr = kstp[c] + (uint32_t)((ks2 >> 1) * C::kBoxBytes) +
                                                  (uint32_t)((nt * 8 + lr) * 128) +
                                                  (((uint32_t)(4 * (ks2 & 1)) ^ kx) << 4);
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(addr, b0, b1, b2, b3);
                            const int k0 = 2 * ks2, k1 = 2 * ks2 + 1;
                            M::mma(sc[c][nt][0], qa[k0][0], qa[k0][1], qa[k0][2], qa[k0][3], b0, b1);
                            M::mma(sc[c][nt][1], qa[k1][0], qa[k1][1], qa[k1][2], qa[k1][3], b2, b3);
                        }
                    }
                }
                // logits of the 32 keys: chunk c, keys c2, c2+1, 8+c2, 9+c2 at [4c .. 4c+3]
                float f[16];  // rows g, then g + 8
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = i >> 2, nt = i >> 1 & 1, e = i & 1;
                    f[i] = sc[c][nt][0][e] + sc[c][nt][1][e];
                    f[8 + i] = sc[c][nt][0][2 + e] + sc[c][nt][1][2 + e];
                }
                to_log2(f);
                float x0[8], x1[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x0[i] = f[i];
                    x1[i] = f[8 + i];
                }
                if (a.slopes) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int key = kb + 16 * (i >> 2) + 8 * (i >> 1 & 1) + c2 + (i & 1);
                        x0[i] -= s0 * fabsf((float)(pos0 - key));
                        x1[i] -= s1 * fabsf((float)(pos1 - key));
                    }
                }
                float mx0 = x0[0], mx1 = x1[0];
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    mx0 = fmaxf(mx0, x0[i]);
                    mx1 = fmaxf(mx1, x1[i]);
                }
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)) - kWeightLift<T>;
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)) - kWeightLift<T>;
                if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
                    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
                    const float al0 = mn0 == -INFINITY ? 1.f : ex2(m0 - mn0);
                    const float al1 = mn1 == -INFINITY ? 1.f : ex2(m1 - mn1);
                    l0 *= al0;
                    l1 *= al1;
#pragma unroll
                    for (int nt = 0; nt < C::kNT; ++nt) {
                        o[nt][0] *= al0;
                        o[nt][1] *= al0;
                        o[nt][2] *= al1;
                        o[nt][3] *= al1;
                    }
                    m0 = mn0;
                    m1 = mn1;
                }
                const float mu0 = m0 == -INFINITY ? 0.f : m0;
                const float mu1 = m1 == -INFINITY ? 0.f : m1;
                float p0[8], p1[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p0[i] = ex2(x0[i] - mu0);
                    p1[i] = ex2(x1[i] - mu1);
                }
                l0 += ((p0[0] + p0[1]) + (p0[2] + p0[3])) + ((p0[4] + p0[5]) + (p0[6] + p0[7]));
                l1 += ((p1[0] + p1[1]) + (p1[2] + p1[3])) + ((p1[4] + p1[5]) + (p1[6] + p1[7]));
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c == 1) {  // the second chunk's V fragments, over the first chunk's
#pragma unroll
                        for (int ntp = 0; ntp < C::kNT / 2; ++ntp) {
                            const uint32_t addr = kstp[1] + C::kTileBytes + (uint32_t)((ntp >> 2) * C::kBoxBytes) +
                                                  (uint32_t)(((lm & 1) * 8 + lr) * 128) +
                                                  (((uint32_t)(2 * (ntp & 3)) ^ vx) << 4);
                            ldsm_x4_t(addr, bv[ntp][0], bv[ntp][1], bv[ntp][2], bv[ntp][3]);
                        }
                    }
                    const uint32_t h0a = M::pack(p0[4 * c], p0[4 * c + 1]), h1a = M::pack(p1[4 * c], p1[4 * c + 1]);
                    const uint32_t h0b = M::pack(p0[4 * c + 2], p0[4 * c + 3]);
                    const uint32_t h1b = M::pack(p1[4 * c + 2], p1[4 * c + 3]);
                    const float2 f0a = M::unpack(h0a), f1a = M::unpack(h1a);
                    const float2 f0b = M::unpack(h0b), f1b = M::unpack(h1b);
                    const uint32_t l0a = M::pack(p0[4 * c] - f0a.x, p0[4 * c + 1] - f0a.y);
                    const uint32_t l1a = M::pack(p1[4 * c] - f1a.x, p1[4 * c + 1] - f1a.y);
                    const uint32_t l0b = M::pack(p0[4 * c + 2] - f0b.x, p0[4 * c + 3] - f0b.y);
                    const uint32_t l1b = M::pack(p1[4 * c + 2] - f1b.x, p1[4 * c + 3] - f1b.y);
#pragma unroll
                    for (int ntq = 0; ntq < C::kNT / 4; ++ntq) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int ntp = 2 * ntq + u;
                            M::mma(o[4 * ntq + 2 * u], h0a, h1a, h0b, h1b, bv[ntp][0], bv[ntp][1]);
                            M::mma(o[4 * ntq + 2 * u + 1], h0a, h1a, h0b, h1b, bv[ntp][2], bv[ntp][3]);
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int ntp = 2 * ntq + u;
                            M::mma(o[4 * ntq + 2 * u], l0a, l1a, l0b, l1b, bv[ntp][0], bv[ntp][1]);
                            M::mma(o[4 * ntq + 2 * u + 1], l0a, l1a, l0b, l1b, bv[ntp][2], bv[ntp][3]);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty0 + 8 * st);
                    mbar_arrive(empty0 + 8 * st2);
                }
                cons += 2;
                ++j;
                continue;
            }
            if (n1 > 0 && kb < wend && kb + 15 >= wbegin) {
                const uint32_t kst = base + (uint32_t)(st * C::kStageBytes) + (uint32_t)(head * C::kHeadSub);
                const uint32_t vst = kst + C::kTileBytes;
                // V fragments first: they do not depend on P, so their shared-memory
                // latency hides behind S and the softmax instead of stalling P V
                uint32_t bv[C::kNT / 2][4];
#pragma unroll
                for (int ntp = 0; ntp < C::kNT / 2; ++ntp) {
                    const uint32_t addr = vst + (uint32_t)((ntp >> 2) * C::kBoxBytes) +
                                          (uint32_t)(((lm & 1) * 8 + lr) * 128) +
                                          (((uint32_t)(2 * (ntp & 3)) ^ vx) << 4);
                    ldsm_x4_t(addr, bv[ntp][0], bv[ntp][1], bv[ntp][2], bv[ntp][3]);
                }
                // ---- S = Q K^T for 16 tokens (two n-tiles of 8), even / odd k-steps apart
                float sc[2][2][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) sc[nt][hh][0] = sc[nt][hh][1] = sc[nt][hh][2] = sc[nt][hh][3] = 0.f;
#pragma unroll
                for (int ks2 = 0; ks2 < C::kKS / 2; ++ks2) {
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const uint32_t addr = kst + (uint32_t)((ks2 >> 1) * C::kBoxBytes) +
                                              (uint32_t)((nt * 8 + lr) * 128) +
                                              (((uint32_t)(4 * (ks2 & 1)) ^ kx) << 4);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(addr, b0, b1, b2, b3);
                        const int k0 = 2 * ks2, k1 = 2 * ks2 + 1;
                        M::mma(sc[nt][0], qa[k0][0], qa[k0][1], qa[k0][2], qa[k0][3], b0, b1);
                        M::mma(sc[nt][1], qa[k1][0], qa[k1][1], qa[k1][2], qa[k1][3], b2, b3);
                    }
                }
                // ---- logits, masks and online softmax; keys c2, c2+1, 8+c2, 9+c2 of rows g, g+8
                float f[8];  // rows g, then g + 8
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int nt = i >> 1, e = i & 1;
                    f[i] = sc[nt][0][e] + sc[nt][1][e];
                    f[4 + i] = sc[nt][0][2 + e] + sc[nt][1][2 + e];
                }
                bool in0[4], in1[4];
                uint32_t any = 0u;  // the keys that some row of this warp sees
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = kb + 8 * (i >> 1) + c2 + (i & 1);
                    in0[i] = key < kb + n1 && key >= k0.x && key < k0.y;
                    in1[i] = key < kb + n1 && key >= k1.x && key < k1.y;
                    if (!in0[i]) f[i] = 0.f;  // as above
                    if (!in1[i]) f[4 + i] = 0.f;
                    if (in0[i] || in1[i]) any |= 1u << (key - kb);
                }
                // (with no partial rows every row that sees any key sees all of these)
                any = kb < win0 || kb + 16 > win1 ? __reduce_or_sync(0xffffffffu, any) : 0xffffu;
                to_log2(f);
                float x0[4], x1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = kb + 8 * (i >> 1) + c2 + (i & 1);
                    x0[i] = in0[i] ? f[i] - s0 * fabsf((float)(pos0 - key)) : -INFINITY;
                    x1[i] = in1[i] ? f[4 + i] - s1 * fabsf((float)(pos1 - key)) : -INFINITY;
                }
                float mx0 = fmaxf(fmaxf(x0[0], x0[1]), fmaxf(x0[2], x0[3]));
                float mx1 = fmaxf(fmaxf(x1[0], x1[1]), fmaxf(x1[2], x1[3]));
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)) - kWeightLift<T>;
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)) - kWeightLift<T>;
                if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
                    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
                    const float al0 = mn0 == -INFINITY ? 1.f : ex2(m0 - mn0);
                    const float al1 = mn1 == -INFINITY ? 1.f : ex2(m1 - mn1);
                    l0 *= al0;
                    l1 *= al1;
#pragma unroll
                    for (int nt = 0; nt < C::kNT; ++nt) {
                        o[nt][0] *= al0;
                        o[nt][1] *= al0;
                        o[nt][2] *= al1;
                        o[nt][3] *= al1;
                    }
                    m0 = mn0;
                    m1 = mn1;
                }
                // a row with no visible key so far has m = -inf and all logits -inf: weights 0
                const float mu0 = m0 == -INFINITY ? 0.f : m0;
                const float mu1 = m1 == -INFINITY ? 0.f : m1;
                float p0[4], p1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p0[i] = ex2(x0[i] - mu0);
                    p1[i] = ex2(x1[i] - mu1);
                }
                l0 += (p0[0] + p0[1]) + (p0[2] + p0[3]);
                l1 += (p1[0] + p1[1]) + (p1[2] + p1[3]);
                // A fragments of P: a0 row g tokens c2.., a1 row g+8 tokens c2.., a2 / a3 tokens 8+c2..
                const uint32_t h0a = M::pack(p0[0], p0[1]), h1a = M::pack(p1[0], p1[1]);
                const uint32_t h0b = M::pack(p0[2], p0[3]), h1b = M::pack(p1[2], p1[3]);
                const float2 f0a = M::unpack(h0a), f1a = M::unpack(h1a);
                const float2 f0b = M::unpack(h0b), f1b = M::unpack(h1b);
                const uint32_t l0a = M::pack(p0[0] - f0a.x, p0[1] - f0a.y);
                const uint32_t l1a = M::pack(p1[0] - f1a.x, p1[1] - f1a.y);
                const uint32_t l0b = M::pack(p0[2] - f0b.x, p0[3] - f0b.y);
                const uint32_t l1b = M::pack(p1[2] - f1b.x, p1[3] - f1b.y);
                if (any != 0xffffu) keep_seen<C::kNT / 2>(bv, any, c2);
                // ---- O += P_hi V + P_lo V, two 16-column groups at a time so that the
                // two MMAs into one accumulator are four issues apart
#pragma unroll
                for (int ntq = 0; ntq < C::kNT / 4; ++ntq) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int ntp = 2 * ntq + u;
                        M::mma(o[4 * ntq + 2 * u], h0a, h1a, h0b, h1b, bv[ntp][0], bv[ntp][1]);
                        M::mma(o[4 * ntq + 2 * u + 1], h0a, h1a, h0b, h1b, bv[ntp][2], bv[ntp][3]);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int ntp = 2 * ntq + u;
                        M::mma(o[4 * ntq + 2 * u], l0a, l1a, l0b, l1b, bv[ntp][0], bv[ntp][1]);
                        M::mma(o[4 * ntq + 2 * u + 1], l0a, l1a, l0b, l1b, bv[ntp][2], bv[ntp][3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * st);
            ++cons;
        }
        if (timed_out) break;

        // ---- finish this warp's two rows per lane
        float lt0 = l0, lt1 = l1;
        lt0 += __shfl_xor_sync(0xffffffffu, lt0, 1);
        lt0 += __shfl_xor_sync(0xffffffffu, lt0, 2);
        lt1 += __shfl_xor_sync(0xffffffffu, lt1, 1);
        lt1 += __shfl_xor_sync(0xffffffffu, lt1, 2);
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
            const bool vr = rr == 0 ? v0 : v1;
            const int tr = rr == 0 ? t0 : t1;
            const int hr = rr == 0 ? h0 : h1;
            const int2 kr = rr == 0 ? k0 : k1;
            const float lt = rr == 0 ? lt0 : lt1;
            const float mr = rr == 0 ? m0 : m1;
            // the plan writes the zeros of rows with an empty range
            if (!vr || kr.x >= kr.y || p < kr.x / Pt || p > (kr.y - 1) / Pt) continue;
            const size_t row = (size_t)(qs + tr) * a.Hq + hr;
            if (kr.x / Pt == (kr.y - 1) / Pt) {
                const float inv = lt != 0.f ? 1.f / lt : 0.f;
#pragma unroll
                for (int nt = 0; nt < C::kNT; ++nt) {
                    const float y0 = o[nt][2 * rr] * inv, y1 = o[nt][2 * rr + 1] * inv;
                    const size_t at = row * D + nt * 8 + c2;
                    if (a.out16) *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + at) = M::pack(y0, y1);
                    else *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(y0, y1);
                }
            } else {
                const size_t r = row * a.max_parts + p;
                float *acc = a.ws_acc + r * D;
#pragma unroll
                for (int nt = 0; nt < C::kNT; ++nt)
                    *reinterpret_cast<float2 *>(acc + nt * 8 + c2) = make_float2(o[nt][2 * rr], o[nt][2 * rr + 1]);
                if ((lane & 3) == 0) *reinterpret_cast<float2 *>(a.ws_ml + 2 * r) = make_float2(mr, lt);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty0 + 8 * slot);  // this warp is done with the item slot
    }
}

template <typename T, int D, int HG, int RW>
cudaError_t launch_scored_chunk_t(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                  cudaStream_t st) {
    using C = ChunkCfg<D, HG, RW>;
    static std::atomic<int> grid_for[kMaxLaunchDevices];
    int grid = 0;
    cudaError_t e = per_device_value(grid_for, &grid, [](int dev, int *v) {
        cudaError_t r = cudaFuncSetAttribute(scored_chunk_kernel<T, D, HG, RW>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (r != cudaSuccess) return r;
        int sms = 0, per_sm = 0;
        r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (r != cudaSuccess) return r;
        r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, scored_chunk_kernel<T, D, HG, RW>, C::kThreads,
                                                          C::kSmem);
        if (r != cudaSuccess) return r;
        *v = sms * (per_sm > 0 ? per_sm : 1);
        return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_chunk_kernel<T, D, HG, RW>, a, tmk, tmv);
}

template <typename T, int D>
cudaError_t dispatch_scored_chunk_d(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    const bool two = a.row_warps == 2;
    switch (a.head_group) {
        case 4: return two ? launch_scored_chunk_t<T, D, 4, 2>(a, tmk, tmv, st) : launch_scored_chunk_t<T, D, 4, 1>(a, tmk, tmv, st);
        case 2: return two ? launch_scored_chunk_t<T, D, 2, 2>(a, tmk, tmv, st) : launch_scored_chunk_t<T, D, 2, 1>(a, tmk, tmv, st);
        case 1: return two ? launch_scored_chunk_t<T, D, 1, 2>(a, tmk, tmv, st) : launch_scored_chunk_t<T, D, 1, 1>(a, tmk, tmv, st);
        default: return cudaErrorNotSupported;
    }
}

template <typename T>
cudaError_t dispatch_scored_chunk(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    if (a.D == 64) return dispatch_scored_chunk_d<T, 64>(a, tmk, tmv, st);
    if (a.D == 128) return dispatch_scored_chunk_d<T, 128>(a, tmk, tmv, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
