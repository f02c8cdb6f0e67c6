// pa_decode_scored.cuh -- scored decode for f16 / bf16 caches on the tensor cores.
//
// For sequence s, query head h and the keys j of the row's range [begin, end),
//   z_j = cap(scale q.k_j) - slope_h (pos - j),  out = sum_j softmax(z)_j v_j,
// with z in log2 units and, when sums are asked for, every z_j left in the
// workspace for the last launch (pa_scored_finish.cu).
//
// Work: an item is (sequence, piece of its range, group of HG KV heads).  The kernel is persistent, two CTAs per SM; a producer warp
// claims items (largest first) and streams their 16-key chunks into a ring of
// shared-memory stages with TMA (one 3-D box is 16 rows of HG heads, 8 KB at HG =
// 4), starting at the 16-key chunk that holds the range's first key, so a window or a
// document costs only the chunks it touches.  Consumer warp w computes KV head
// g0 + w: S = Q K^T and O += P V with mma.m16n8k16, the G <= 8 query heads as
// rows 0-7 of A; for P V rows 0-7 carry the weights' high 16-bit part and rows
// 8-15 the low part, so that weights keep 16 (bf16) or 22 (f16) bits; the running
// maximum m is held 15 octaves below the largest logit for f16 (kWeightLift).
// Keys outside the range get -inf and their V rows are zeroed in shared
// memory, so what they hold does not matter.
//
// Bound: HBM (4 D bytes per key and KV head against G x 4 D flops).
// Measured (D 128): 256 sequences, 32 / 8 heads, bf16, capped 126 us = 6.7 TB/s, 146 with sums; 64
// sequences, 32 / 32 heads, f16, documents and bias 114 us (floor 113); a window of 4096 over 32 long
// sequences, 64 / 8 heads, bf16, 89 us, 107 with sums (floor 78, 80).
#pragma once

#include <cuda.h>

#include <cmath>

#include "pa_mma.cuh"
#include "pa_score.cuh"

namespace pa {

template <int D, int HG>
struct ScoredDecodeCfg {
    static constexpr int kKS = D / 16;                   // k-steps of q.k
    static constexpr int kNT = D / 8;                    // 8-wide n-tiles of p.v
    static constexpr int kSub = D / 64;                  // 128-byte halves of a row
    static constexpr int kHeadSub = 16 * 128;            // one head's half-rows of a chunk
    static constexpr int kBoxBytes = HG * kHeadSub;      // one TMA box: that, for HG heads
    static constexpr int kTileBytes = kSub * kBoxBytes;  // K (or V) of a chunk, all HG heads
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kThreads = (HG + 1) * 32;       // consumer warps + the producer
    static constexpr int kStagesRaw = 96 * 1024 / kStageBytes;
    static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
    static constexpr int kSlots = 3;                     // work items in flight per CTA
    static constexpr size_t kFullOff = (size_t)kStages * kStageBytes;
    static constexpr size_t kEmptyOff = kFullOff + 8 * kStages;
    static constexpr size_t kItemFullOff = kEmptyOff + 8 * kStages;
    static constexpr size_t kItemEmptyOff = kItemFullOff + 8 * kSlots;
    static constexpr size_t kInfoOff = kItemEmptyOff + 8 * kSlots;  // kSlots x (s, piece, lo, hi), (g0, chunks, valid, pos)
    static constexpr size_t kTblOff = kInfoOff + 32 * kSlots;
    static constexpr size_t kSmem = kTblOff + (size_t)kSlots * kMaxPartitionBlocks * 4 + 1024;  // + alignment slack
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(kStages >= 2, "ring");
    static_assert(kHeadSub % 1024 == 0, "swizzle atoms must stay 1024-byte aligned");
    static_assert(kInfoOff % 16 == 0, "int4 slot info");
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
};

template <typename T, int D, int HG>
__global__ void __launch_bounds__(ScoredDecodeCfg<D, HG>::kThreads, 2)
    scored_decode_kernel(const ScoredArgs a, const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv) {
    using C = ScoredDecodeCfg<D, HG>;
    using M = Mma16<T>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // the 128-byte swizzle repeats every 1 KB
    unsigned char *basep = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv;
    const int ngroups = a.Hkv / HG;
    const int cap = a.max_blocks * a.B;

    const uint32_t full0 = base + (uint32_t)C::kFullOff;
    const uint32_t empty0 = base + (uint32_t)C::kEmptyOff;
    const uint32_t ifull0 = base + (uint32_t)C::kItemFullOff;
    const uint32_t iempty0 = base + (uint32_t)C::kItemEmptyOff;
    int4 *info = reinterpret_cast<int4 *>(basep + C::kInfoOff);
    int32_t *tbl = reinterpret_cast<int32_t *>(basep + C::kTblOff);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, HG);
        }
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(ifull0 + 8 * i, 1);
            mbar_init(iempty0 + 8 * i, HG);
        }
        fence_mbar_init();
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    __syncthreads();
    // The plan released this grid after everything before it had completed: the
    // caches, tables, lengths and masks may be read; only the list needs the plan.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == HG) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = policy_evict_first();
        const int nstatic = min(a.S, (int)gridDim.x / ngroups) * ngroups;  // items taken without the list
        const int lb = __ffs(a.B) - 1;  // block_size is a power of two
        bool listed = false;
        int n_items = 0;
        int iss = 0;  // chunks issued
        bool ok = true;
        for (int seq = 0; ok; ++seq) {
            const int slot = seq % C::kSlots;
            if (seq >= C::kSlots &&
                !mbar_wait_bounded(iempty0 + 8 * slot, (uint32_t)((seq / C::kSlots) - 1) & 1u, kWaitLimit)) {
                if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                break;
            }
            int4 e = make_int4(0, 0, 0, 0);
            int g0 = 0;
            bool have = false;
            if (seq == 0 && (int)blockIdx.x < nstatic) {
                const int s = blockIdx.x / ngroups;
                const RowOf r = row_of(a, s, cap);
                const int2 k = row_range(a, s, r.pos, r.len);
                if (k.x < k.y) {
                    const int2 p = piece_of(k, a.partition_size, a.partition_size, 0);  // the same for every plan
                    e = make_int4(s, p.y == k.y ? kWholeRange : 0, p.x, p.y);
                    g0 = (blockIdx.x % ngroups) * HG;
                    have = true;
                }
            }
            if (!have) {
                if (!listed) {
                    griddep_wait();
                    n_items = a.plan_hdr[0];
                    listed = true;
                }
                // CTAs past the directly taken items start with list entry
                // b - nstatic, without an atomic; later claims follow them
                int idx = 0;
                if (seq == 0 && (int)blockIdx.x >= nstatic) idx = blockIdx.x - nstatic;
                else if (lane == 0) idx = (int)gridDim.x - nstatic + atomicAdd(a.plan_hdr + 1, 1);
                idx = __shfl_sync(0xffffffffu, idx, 0);
                if (idx < n_items) {
                    e = a.plan_list[idx / ngroups];
                    g0 = (idx % ngroups) * HG;
                    have = true;
                }
            }
            const int k16 = e.z & ~15;  // first key of the first chunk
            const int nchunk = have ? (e.w - k16 + 15) >> 4 : 0;
            int32_t *tb = tbl + slot * kMaxPartitionBlocks;
            const int blk0 = k16 >> lb;
            if (have) {
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
                int pos = 0;
                if (have) {
                    const int len = a.context_lens[e.x];
                    pos = (len > cap ? cap : len) - 1;
                }
                info[2 * slot] = e;
                info[2 * slot + 1] = make_int4(g0, nchunk, have ? 1 : 0, pos);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ifull0 + 8 * slot);  // release: info and table visible
            if (!have) break;
            for (int c = 0; c < nchunk; ++c) {
                const int st = iss % C::kStages;
                if (iss >= C::kStages &&
                    !mbar_wait_bounded(empty0 + 8 * st, (uint32_t)((iss / C::kStages) - 1) & 1u, kWaitLimit)) {
                    if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t bar = full0 + 8 * st;
                    const int key = k16 + 16 * c;
                    const int pb = tb[(key >> lb) - blk0];
                    if (pb < 0) {
                        mbar_arrive(bar);  // bad table entry: complete the phase without data
                    } else {
                        const uint32_t dst = base + (uint32_t)(st * C::kStageBytes);
                        const int y = key & (a.B - 1);
                        const int z = pb * a.Hkv + g0;
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
        // the CTA's shared memory outlives its copies
        for (int k = iss > C::kStages ? iss - C::kStages : 0; k < iss; ++k)
            mbar_wait_bounded(full0 + 8 * (k % C::kStages), (uint32_t)(k / C::kStages) & 1u, kWaitLimit);
        // no CTA of this grid ends before the plan has: whatever waits for this grid waits for both
        if (!listed) griddep_wait();
        return;
    }

    // ------------------------------------------------------------ consumer warps
    const int g = lane >> 2;         // fragment row = query head within the group (rows 8-15: low parts)
    const int c2 = (lane & 3) * 2;   // fragment column pair
    const int lm = lane >> 3;        // ldmatrix: which 8x8 matrix this lane addresses
    const int lr = lane & 7;         // ldmatrix: which row of it
    const uint32_t kx = (uint32_t)(lm ^ lr);          // swizzled chunk bits for K reads
    const uint32_t vx = (uint32_t)((lm >> 1) ^ lr);   // and for V reads
    const ScoreCap score(a);
    uint32_t qa[C::kKS][2];
    int cons = 0;  // chunks consumed by this warp
    for (int seq = 0;; ++seq) {
        const int slot = seq % C::kSlots;
        if (!mbar_wait_bounded(ifull0 + 8 * slot, (uint32_t)(seq / C::kSlots) & 1u, kWaitLimit)) {
            if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
            break;
        }
        const int4 e0 = info[2 * slot];
        const int4 e1 = info[2 * slot + 1];
        if (!e1.z) break;  // no more work
        const int s = e0.x, p = e0.y & ~kWholeRange, lo = e0.z, hi = e0.w;
        const bool whole = (e0.y & kWholeRange) != 0;
        const int k16 = lo & ~15;
        const int kvh = e1.x + warp;
        const int nchunk = e1.y, pos = e1.w;
        const int h = kvh * G + g;
        const int32_t *ctb = tbl + slot * kMaxPartitionBlocks;
        const int lb = __ffs(a.B) - 1, blk0 = k16 >> lb;
        const uint16_t *qrow = static_cast<const uint16_t *>(a.q) + ((size_t)s * a.Hq + h) * D;
#pragma unroll
        for (int ks = 0; ks < C::kKS; ++ks) {
            qa[ks][0] = g < G ? *reinterpret_cast<const uint32_t *>(qrow + ks * 16 + c2) : 0u;
            qa[ks][1] = g < G ? *reinterpret_cast<const uint32_t *>(qrow + ks * 16 + 8 + c2) : 0u;
        }
        const float slope = a.slopes && g < G ? a.slopes[h] * kLog2e : 0.f;
        float *lrow = a.ws_logits ? a.ws_logits + ((size_t)s * a.Hq + h) * cap : nullptr;
        float o[C::kNT][4];
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
        float m_run = -INFINITY, l_run = 0.f;
        bool timed_out = false;

        for (int j = 0; j < nchunk; ++j) {
            const int st = cons % C::kStages;
            if (!__all_sync(0xffffffffu,
                            mbar_wait_bounded(full0 + 8 * st, (uint32_t)(cons / C::kStages) & 1u, kWaitLimit))) {
                if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
                timed_out = true;
                break;
            }
            const int kb = k16 + 16 * j;
            const int n0 = max(lo - kb, 0);                                         // keys n0 .. n1 - 1 of the chunk count
            const int n1 = ctb[(kb >> lb) - blk0] < 0 ? 0 : min(16, hi - kb);
            const uint32_t kst = base + (uint32_t)(st * C::kStageBytes) + (uint32_t)(warp * C::kHeadSub);
            const uint32_t vst = kst + C::kTileBytes;
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (n1 > 0) {
                if (n0 > 0 || n1 < 16) {
                    // zero this head's V rows outside the range (whole 128-byte rows: the swizzle does not matter)
                    for (int i = lane; i < 16 * C::kSub * 8; i += 32) {
                        const int r = (i >> 3) & 15;
                        if (r >= n0 && r < n1) continue;
                        const uint32_t addr = vst + (i >> 7) * C::kBoxBytes + r * 128 + (i & 7) * 16;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
                    }
                    __syncwarp();
                }
                // ---- S = Q K^T for 16 keys (two n-tiles of 8), even and odd k-steps apart
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
                                              (uint32_t)((nt * 8 + lr) * 128) + (((uint32_t)(4 * (ks2 & 1)) ^ kx) << 4);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(addr, b0, b1, b2, b3);
                        M::mma(sc[nt][0], qa[2 * ks2][0], 0u, qa[2 * ks2][1], 0u, b0, b1);
                        M::mma(sc[nt][1], qa[2 * ks2 + 1][0], 0u, qa[2 * ks2 + 1][1], 0u, b2, b3);
                    }
                }
                // ---- this lane's row g, keys c2, c2 + 1, c2 + 8, c2 + 9 of the chunk
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = c2 + (i & 1) + 8 * (i >> 1);
                    const float z = score(sc[i >> 1][0][i & 1] + sc[i >> 1][1][i & 1]) - slope * (float)(pos - kb - kk);
                    x[i] = kk >= n0 && kk < n1 ? z : -INFINITY;
                }
            }
            if (lrow && g < G) {
                *reinterpret_cast<float2 *>(lrow + kb + c2) = make_float2(x[0], x[1]);
                *reinterpret_cast<float2 *>(lrow + kb + 8 + c2) = make_float2(x[2], x[3]);
            }
            if (n1 > 0) {
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) - kWeightLift<T>;
                if (__any_sync(0xffffffffu, mx > m_run)) {
                    const float mn = fmaxf(m_run, mx);
                    const float al = mn == -INFINITY ? 1.f : ex2(m_run - mn);
                    l_run *= al;
#pragma unroll
                    for (int nt = 0; nt < C::kNT; ++nt) {
                        o[nt][0] *= al;
                        o[nt][1] *= al;
                        o[nt][2] *= al;
                        o[nt][3] *= al;
                    }
                    m_run = mn;
                }
                const float mu = m_run == -INFINITY ? 0.f : m_run;
                float pr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pr[i] = ex2(x[i] - mu);
                l_run += (pr[0] + pr[1]) + (pr[2] + pr[3]);
                const uint32_t h01 = M::pack(pr[0], pr[1]);
                const uint32_t h23 = M::pack(pr[2], pr[3]);
                const float2 f01 = M::unpack(h01);
                const float2 f23 = M::unpack(h23);
                const uint32_t l01 = M::pack(pr[0] - f01.x, pr[1] - f01.y);
                const uint32_t l23 = M::pack(pr[2] - f23.x, pr[3] - f23.y);
                // ---- O += P V
#pragma unroll
                for (int ntp = 0; ntp < C::kNT / 2; ++ntp) {
                    const uint32_t addr = vst + (uint32_t)((ntp >> 2) * C::kBoxBytes) +
                                          (uint32_t)(((lm & 1) * 8 + lr) * 128) + (((uint32_t)(2 * (ntp & 3)) ^ vx) << 4);
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4_t(addr, b0, b1, b2, b3);
                    M::mma(o[2 * ntp], h01, l01, h23, l23, b0, b1);
                    M::mma(o[2 * ntp + 1], h01, l01, h23, l23, b2, b3);
                }
            }
            // order these generic shared-memory accesses before the next bulk copy into the stage
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * st);
            ++cons;
        }
        if (timed_out) break;

        // ---- finish this warp's head of the item
        float lt = l_run;
        lt += __shfl_xor_sync(0xffffffffu, lt, 1);
        lt += __shfl_xor_sync(0xffffffffu, lt, 2);
        if (g < G) {
            const size_t r = ((size_t)s * a.Hq + h) * a.max_parts + p;
            if (whole) {
                const float inv = lt != 0.f ? 1.f / lt : 0.f;
                const size_t at = ((size_t)s * a.Hq + h) * D + c2;
#pragma unroll
                for (int nt = 0; nt < C::kNT; ++nt) {
                    const float y0 = (o[nt][0] + o[nt][2]) * inv, y1 = (o[nt][1] + o[nt][3]) * inv;
                    if (a.out16) *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + at + nt * 8) = M::pack(y0, y1);
                    else *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at + nt * 8) = make_float2(y0, y1);
                }
            } else {
                float *acc = a.ws_acc + r * D + c2;
#pragma unroll
                for (int nt = 0; nt < C::kNT; ++nt)
                    *reinterpret_cast<float2 *>(acc + nt * 8) = make_float2(o[nt][0] + o[nt][2], o[nt][1] + o[nt][3]);
            }
            if ((!whole || a.ws_logits) && (lane & 3) == 0)
                *reinterpret_cast<float2 *>(a.ws_ml + 2 * r) = make_float2(m_run, lt);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty0 + 8 * slot);  // this warp is done with the item slot
    }
}

template <typename T, int D, int HG>
cudaError_t scored_decode_grid_t(int *grid) {
    using C = ScoredDecodeCfg<D, HG>;
    static std::atomic<int> grid_for[kMaxLaunchDevices];
    return per_device_value(grid_for, grid, [](int dev, int *v) {
        cudaError_t e = cudaFuncSetAttribute(scored_decode_kernel<T, D, HG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)C::kSmem);
        if (e != cudaSuccess) return e;
        int sms = 0, per_sm = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, scored_decode_kernel<T, D, HG>, C::kThreads, C::kSmem);
        if (e != cudaSuccess) return e;
        *v = sms * (per_sm > 0 ? per_sm : 1);
        return cudaSuccess;
    });
}

template <typename T, int D, int HG>
cudaError_t launch_scored_decode_t(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    using C = ScoredDecodeCfg<D, HG>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_decode_kernel<T, D, HG>, a, tmk, tmv);
}

// Calls f with the (D, HG) pair of the launch as compile-time constants.
template <typename F>
cudaError_t with_scored_shape(const ScoredArgs &a, F f) {
    using std::integral_constant;
    if (a.D != 64 && a.D != 128) return cudaErrorNotSupported;
    switch (a.head_group) {
        case 4: return a.D == 64 ? f(integral_constant<int, 64>(), integral_constant<int, 4>())
                                 : f(integral_constant<int, 128>(), integral_constant<int, 4>());
        case 2: return a.D == 64 ? f(integral_constant<int, 64>(), integral_constant<int, 2>())
                                 : f(integral_constant<int, 128>(), integral_constant<int, 2>());
        case 1: return a.D == 64 ? f(integral_constant<int, 64>(), integral_constant<int, 1>())
                                 : f(integral_constant<int, 128>(), integral_constant<int, 1>());
        default: return cudaErrorNotSupported;
    }
}

template <typename T>
cudaError_t dispatch_scored_decode(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    return with_scored_shape(a, [&](auto d, auto hg) {
        return launch_scored_decode_t<T, decltype(d)::value, decltype(hg)::value>(a, tmk, tmv, st);
    });
}

template <typename T>
cudaError_t dispatch_scored_decode_ctas(const ScoredArgs &a, int *ctas) {
    return with_scored_shape(a, [&](auto d, auto hg) {
        return scored_decode_grid_t<T, decltype(d)::value, decltype(hg)::value>(ctas);
    });
}

}  // namespace pa
