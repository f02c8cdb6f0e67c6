// pa_chunk_scored_umma.cuh -- scored chunk attention for long query chunks on
// the 5th-generation tensor cores (tcgen05.mma, accumulators in tensor memory).
//
// For the query row at position pos and the keys j of its own range [begin, end)
//   z_j = cap(scale q.k_j) - slope_h |pos - j|,   out = sum_j softmax(z)_j v_j.
// The structure is that of the plain long-chunk kernel (pa_chunk_umma.cuh, whose
// tile configuration and barrier helpers this file uses): persistent CTAs that
// claim (two 128-row tiles, KV head, sequence) items longest first, warps 0 and 2
// streaming K and V by TMA in steps of 64 keys, one warp per tile issuing S = Q
// K^T and one issuing O += P V with P = P_hi + P_lo taken from tensor memory, and
// one softmax warpgroup per tile, one thread per row.
//
// What differs: an item walks the 64-key steps from the first key that some of its
// rows sees to the last, so a document or a window costs only its own steps; 16-row
// boxes outside that span are not loaded; each row masks to its own range (steps
// that every row of a warp sees whole skip the test); cap and bias are
// applied to the logits in registers; V rows that no row of the item sees are zeroed (by the softmax outside
// the item's span, by the P V issuers in holes between the rows' ranges, for the items that the plan marks);
// the output may be 16-bit, staged in the query tile's own layout and stored by
// TMA with a map like the queries'.
//
// Bound: a step's chain from S through the softmax to P V.  Measured (the kernel alone), 16 x 512-token chunks over
// contexts of up to 4096 (32 / 8 heads, D 128, bf16): ranges only 255 us, bias 314, cap 319 (753 TFLOP/s of the 4 D
// flops a key and head), both 465; f16, cap 358; D 64, cap 297; the tensor cores' own time would be 127 us, 191 with
// the low parts' products.  Of the 319 capped, 148 are left without the softmax's arithmetic (cap, masks, exponentials,
// split) and without the products, 210 without the arithmetic, 278 without the products: about half is the
// roles' waiting for each other, and most of the rest the arithmetic, which the products only partly hide.
// Ragged prompts with a prefix mask and a bias (D 64, f16) 58 us.  Tried and slower, against the time of
// then: two threads a row (sixteen softmax warps, 329 -> 344 us), S and P in columns of their own (329 -> 341);
// P V of the two tiles issued one whole step after the other: 318 -> 308, but f16 354 -> 364 and D 64 296 -> 307.
#pragma once

#include <cuda.h>

#include <cmath>
#include <type_traits>

#include "pa_chunk_umma.cuh"
#include "pa_score.cuh"

namespace pa {

// What a kernel's softmax does to the logits, fixed at compile time so that the
// others' state takes no registers in the loop (at most 128 a thread).  All but
// kGeneral need a positive scale.
enum ScoredMode {
    kMaskOnly,   // ranges only
    kCapFixed,   // bf16, cap of at most 55: no running maximum (see below)
    kCapMax,     // cap, running maximum
    kBias,       // distance bias
    kGeneral,    // cap and bias, or a scale that is not positive
};
inline ScoredMode scored_mode(const ScoredArgs &a, bool bf16) {
    if (!(a.scale > 0.f) || (a.softcap > 0.f && a.slopes)) return kGeneral;
    if (a.slopes) return kBias;
    if (a.softcap > 0.f) return bf16 && a.softcap * kLog2e <= 80.f ? kCapFixed : kCapMax;
    return kMaskOnly;
}

// Bits 0 .. x - 1 of a word (none for x <= 0, all from 32 on).
__device__ __forceinline__ uint32_t bits_below(int x) { return x >= 32 ? ~0u : (1u << max(x, 0)) - 1u; }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The plain kernel's tiles and shared memory.  With two tiles and logits that are capped or
// biased, the softmax warpgroups come behind two whole warpgroups of producers and issuers (two
// warps of which idle), so that the latter's registers can be handed to them: 512 threads
// are launched at 128 registers, 8 warps keep 72 and 8 take 184 (8 x 72 + 8 x 184 = 16 x 128).
// Measured on 16 x 512-token chunks of D 128: capped 356 -> 350 us, both 508 -> 486, ragged
// biased prompts of D 64 69 -> 65; with ranges only 260 -> 268, so that kernel keeps the 14 warps.
template <int D, int MT, int kMode>
struct ScoredUmmaCfg : UmmaCfg<D, MT> {
    static constexpr bool kRegSplit = MT == 2 && kMode != kMaskOnly;
    static constexpr int kSoftWarp0 = kRegSplit ? 8 : UmmaCfg<D, MT>::kSoftWarp0;
    static constexpr int kThreads = 32 * (kSoftWarp0 + 4 * MT);
    // boxes loaded of the last kMasks steps, in place of the plain kernel's per ring stage
    static constexpr int kMasks = 16;
    static constexpr size_t kMasksOff = (UmmaCfg<D, MT>::kItemOff + (size_t)MT * 2 * 64 + 7) / 8 * 8;
    static constexpr size_t kZeroedOff = kMasksOff + 4 * kMasks;  // a barrier per entry
    static constexpr size_t kSmem = UmmaCfg<D, MT>::kSmem + 8 + (4 + 8) * kMasks;
    static_assert(kZeroedOff % 8 == 0, "barriers");
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// One work item: KV head kvh of the plan's entry (sequence s, tile group), i.e.
// rows r0 .. r0 + 128 MT - 1 of that head's (query token, query head) rows, and
// the keys [lo, hi) from the first to the last that some of those rows see, in nch steps.
// s carries kHoles too: whether there may be keys among them that no row sees.
struct ScoredItem {
    int s, kvh, r0, qs, n, len, tiles, nch, lo, hi;
};
// A work item as the K producer publishes it to a tile's roles, or the end
// mark (no more items).
struct ScoredSlot {
    ScoredItem it;
    int end;
};
static_assert(sizeof(ScoredSlot) <= 64, "a slot's share of shared memory");

// Work index w = entry * Hkv + kvh of the plan's longest-first list; false past its end.
template <typename C>
__device__ __forceinline__ bool scored_item(const ScoredArgs &a, int w, int nwork, ScoredItem &it) {
    if (w >= nwork) return false;
    const int4 e = a.plan_list[w / a.Hkv];  // (sequence, tile group, first key, one past the last)
    const int G = a.Hq / a.Hkv;
    const int s = e.x & ~kHoles;
    it.s = e.x;
    it.kvh = w % a.Hkv;
    it.r0 = e.y * C::kM * C::kMT;
    it.qs = a.query_start[s];
    it.n = a.query_start[s + 1] - it.qs;
    it.len = a.context_lens[s];
    it.tiles = min(C::kMT, (it.n * G - it.r0 + C::kM - 1) / C::kM);  // tiles with at least one row
    it.lo = e.z;
    it.hi = e.w;
    it.nch = (e.w - 1) / C::kN - e.z / C::kN + 1;
    return true;
}

// The ring's stage and phase follow the count g of steps so far, the S/P buffers
// and their phases the count c of the tile's own steps, the slots and query-tile
// sets the count of items published.
template <typename T, int D, int MT, int kMode>
__global__ void __launch_bounds__(ScoredUmmaCfg<D, MT, kMode>::kThreads, 1)
    scored_umma_kernel(const ScoredArgs a, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmo) {
    using C = ScoredUmmaCfg<D, MT, kMode>;
    using M = Mma16<T>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *basep = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    const int G = a.Hq / a.Hkv;

    const uint32_t qb = base + (uint32_t)C::kQOff;
    const uint32_t kvb = base + (uint32_t)C::kKVOff;
    const uint32_t bars = base + (uint32_t)C::kBarOff;
    auto k_full = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto k_empty = [&](int i) { return bars + 8u * (uint32_t)(C::kStages + i); };
    auto v_full = [&](int i) { return bars + 8u * (uint32_t)(2 * C::kStages + i); };
    auto v_empty = [&](int i) { return bars + 8u * (uint32_t)(3 * C::kStages + i); };
    // Tile 0's softmax has zeroed the V rows of step g that must not contribute.  A ring of kMasks, not of
    // stages: tile 0 publishes step g once P V of g - kSB is done, so once the other tile's P V of g - kSB - kStages
    // has released its V; with kStages barriers it could complete one twice before that tile has seen it once.
    auto v_zeroed = [&](int g) { return base + (uint32_t)(C::kZeroedOff + 8 * (g % C::kMasks)); };
    auto tbar = [&](int u, int i) { return bars + 8u * (uint32_t)(5 * C::kStages + u * C::kTileBars + i); };
    constexpr int kSB = C::kSB;
    auto s_full = [&](int u, int b) { return tbar(u, b); };
    auto p_full = [&](int u, int b) { return tbar(u, kSB + b); };
    // P V of a step on buffer b complete: O is up to date and S/P[u][b] may be rewritten
    auto o_done = [&](int u, int b) { return tbar(u, 2 * kSB + b); };
    auto q_full = [&](int u, int x) { return tbar(u, 3 * kSB + x); };
    // the epilogue has finished with query-tile set x of tile u (its staging area)
    auto q_free = [&](int u, int x) { return tbar(u, 3 * kSB + 2 + x); };
    auto drain_s = [&](int u) { return tbar(u, 3 * kSB + 4); };
    auto drain_p = [&](int u) { return tbar(u, 3 * kSB + 5); };
    // the K producer has published tile u's next item in slot x
    auto item_ready = [&](int u, int x) { return tbar(u, 3 * kSB + 6 + x); };
    ScoredSlot *slots = reinterpret_cast<ScoredSlot *>(basep + C::kItemOff);
    auto slot = [&](int u, int x) -> ScoredSlot & { return slots[2 * u + x]; };
    // wait for tile u's k-th published item (slot k & 1) and read it
    auto take = [&](int u, int k, ScoredSlot &out) {
        const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(item_ready(u, k & 1), (uint32_t)(k >> 1) & 1u, kWaitLimit));
        if (got) out = slot(u, k & 1);
        __syncwarp();  // every lane has read it before one of them frees the slot
        return got;
    };
    auto qtile = [&](int x, int u) { return qb + (uint32_t)((x * MT + u) * C::kQTile); };
    auto s_col = [&](int u, int b) { return (uint32_t)(128 * u + C::kN * b); };
    auto o_col = [&](int u) { return C::kOCol + (uint32_t)(D * u); };
    // Boxes loaded of step g.  The K producer writes it before the step's K lands, so that a tile that has
    // seen S knows it.  It writes step g once S of g - kStages is done, so tile 0's P V of kSB steps before, whose V
    // came when both tiles' P V had released that of kStages before: every tile has read what lies
    // 2 kStages + kSB steps back (8; 16 with steps of 32 keys).  So the softmax waits for V only where it zeroes
    // rows of it (waiting in every step: 325 us against 319 on 16 x 512-token capped chunks).
    int *masks = reinterpret_cast<int *>(basep + C::kMasksOff);
    auto zero_v_row = [&](uint32_t row) {  // both halves of a row of a step's V
#pragma unroll
        for (int sb = 0; sb < C::kSub; ++sb)
#pragma unroll
            for (int cc = 0; cc < 8; ++cc)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(row + sb * C::kHalf + cc * 16), "r"(0u) : "memory");
    };
    static_assert(2 * C::kStages + C::kSB <= C::kMasks, "a mask must outlive its readers");
    uint32_t *tslot = reinterpret_cast<uint32_t *>(basep + C::kSlotOff);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(k_empty(i), MT);  // one arrival per tile's S issuer (a commit, or a plain
            mbar_init(v_full(i), 1);    // arrival when the item has no rows in that tile)
            mbar_init(v_empty(i), MT);  // likewise from each tile's P V issuer
        }
        for (int i = 0; i < C::kMasks; ++i) mbar_init(v_zeroed(i), 4);
        for (int u = 0; u < MT; ++u) {
            for (int b = 0; b < kSB; ++b) {
                mbar_init(s_full(u, b), 1);
                mbar_init(p_full(u, b), 4);
                mbar_init(o_done(u, b), 1);
            }
            for (int x = 0; x < 2; ++x) {
                mbar_init(q_full(u, x), 1);
                mbar_init(q_free(u, x), 4 + 2);  // the softmax warps, and both MMA issuers once they have read the slot
                mbar_init(item_ready(u, x), 1);
            }
            mbar_init(drain_s(u), 1);
            mbar_init(drain_p(u), 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmo);
    }
    if (warp == 1) tc::tmem_alloc(smem_addr(tslot), C::kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    griddep_wait();  // the plan kernel's list of (sequence, tile group), longest first
    const int nwork = a.plan_hdr[0] > 0 ? a.plan_hdr[0] * a.Hkv : 0;

    if (warp < C::kSoftWarp0) {
    if constexpr (C::kRegSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n" ::: "memory");
    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers: K (warp 0), V (warp 2)
        const bool is_v = warp == 2;
        const uint64_t pol = policy_evict_last();  // the other row tiles of this head reread these keys
        const uint64_t qpol = policy_evict_first();
        const CUtensorMap *map = is_v ? &tmv : &tmk;
        const uint32_t ring = kvb + (is_v ? (uint32_t)C::kTile : 0u);
        const int bx = lane % C::kBoxes, sbx = lane / C::kBoxes;
        int g = 0;                  // ring steps issued
        int ku[MT];                 // items published to each tile so far (query-tile sets)
#pragma unroll
        for (int u = 0; u < MT; ++u) ku[u] = 0;
        int k0 = 0;                 // V producer: tile 0's items taken so far
        int items = 0;              // K producer: entries taken so far
        bool ok = true;
        for (;;) {
            ScoredItem it;
            if (!is_v) {
                // claim the next entry of the longest-first list; past its end, publish the
                // end mark to every tile
                int w = blockIdx.x;  // a CTA's first entry needs no claim
                if (items++ > 0) {
                    if (lane == 0) w = (int)gridDim.x + atomicAdd(&a.plan_hdr[1], 1);
                    w = __shfl_sync(0xffffffffu, w, 0);
                }
                const bool have = scored_item<C>(a, w, nwork, it);
                // every tile's roles see every item (a tile without rows in it releases
                // its ring stages); slot x of tile u is free once the tile's roles are
                // done with the item before last
                for (int u = 0; ok && u < MT; ++u) {
                    const int x = ku[u] & 1;
                    if (ku[u] >= 2) ok = mbar_wait_bounded(q_free(u, x), (uint32_t)((ku[u] >> 1) - 1) & 1u, kWaitLimit);
                    if (ok && lane == 0) {
                        ScoredSlot &sl = slot(u, x);
                        if (have) sl.it = it;
                        sl.end = have ? 0 : 1;
                        mbar_arrive(item_ready(u, x));
                        if (have && u >= it.tiles) {
                            mbar_arrive(q_full(u, x));  // no query tile: keep the set's phases in step
                        } else if (have) {
                            // the query tile: tile u holds rows r0 + 128 u .., i.e. tokens
                            // (r0 + 128 u) / G .. of the sequence's chunk, G heads each; rows
                            // of tokens past the chunk are never used (their keys are all masked)
                            mbar_arrive_expect_tx(q_full(u, x), (uint32_t)C::kQTile);
#pragma unroll
                            for (int sb = 0; sb < C::kSub; ++sb)
                                tma_load_3d(qtile(x, u) + (uint32_t)(sb * C::kQHalf), &tmq, sb * 64, it.kvh * G,
                                            it.qs + (it.r0 + C::kM * u) / G, q_full(u, x), qpol);
                        }
                    }
                    ++ku[u];
                }
                __syncwarp();
                if (!ok || !have) break;
            } else {
                // the V producer follows tile 0's items (tile 0 has rows in every item)
                ScoredSlot sl;
                ok = take(0, k0++, sl);
                if (!ok || sl.end) break;
                it = sl.it;
            }
            // One lane per copy: box bx of 16 keys, 64 of their columns; its block id is read a step
            // ahead.  (One lane reading the four ids and issuing the eight copies in turn held the steps up:
            // 345 us against 329 on 16 x 512-token capped chunks, 280 against 263 with ranges only.)
            const int32_t *row = a.block_tables + (size_t)(it.s & ~kHoles) * a.max_blocks;
            const int j0 = it.lo / C::kN, lb = __ffs(a.B) - 1;  // B is a power of two
            auto wanted = [&](int j) {
                const int tok = j * C::kN + 16 * bx;
                return lane < C::kBoxes * C::kSub && tok + 15 >= it.lo && tok < it.hi;
            };
            int next = wanted(j0) ? row[(j0 * C::kN + 16 * bx) >> lb] : 0;
            for (int j = j0; j < j0 + it.nch; ++j, ++g) {
                const int st = g % C::kStages;
                const int pbk = next, tok = j * C::kN + 16 * bx;
                const bool want = wanted(j), good = want && pbk >= 0 && pbk < a.N;
                if (j + 1 < j0 + it.nch && wanted(j + 1)) next = row[(tok + C::kN) >> lb];
                if (want && !good && !is_v) set_error(a.err, PA_DEVERR_BAD_BLOCK);
                const int mask = (int)(__ballot_sync(0xffffffffu, good) & ((1u << C::kBoxes) - 1u));
                if (g >= C::kStages &&
                    !mbar_wait_bounded(is_v ? v_empty(st) : k_empty(st), (uint32_t)((g / C::kStages) - 1) & 1u,
                                       kWaitLimit)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = is_v ? v_full(st) : k_full(st);
                if (lane == 0) {
                    if (!is_v) masks[g % C::kMasks] = mask;
                    if (mask == 0) mbar_arrive(bar);
                    else mbar_arrive_expect_tx(bar, (uint32_t)__popc(mask) * C::kSub * 2048u);
                }
                __syncwarp();
                if (good)
                    tma_load_3d(ring + (uint32_t)(st * C::kStageBytes + sbx * C::kHalf + bx * 2048), map, sbx * 64,
                                tok & (a.B - 1), pbk * a.Hkv + it.kvh, bar, pol);
                __syncwarp();
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
        // copies still in flight must land before the CTA's shared memory is released
        for (int k = max(0, g - C::kStages); k < g; ++k)
            mbar_wait_bounded(is_v ? v_full(k % C::kStages) : k_full(k % C::kStages), (uint32_t)(k / C::kStages) & 1u,
                              kWaitLimit);
    } else if (warp == 1 || (MT == 2 && warp == 4)) {
        // ------------------------------------------------------------ S = Q K^T issuer of tile u
        // One issuer per tile: a tile waits for its own P V, not the other tile's.
        const int u = warp == 1 ? 0 : 1;
        constexpr uint32_t idesc_s = tc::f16_idesc(kBf16, false, C::kM, C::kN);
        // Descriptors built once: a step's operands are these plus compile-time
        // offsets (tc::desc_add), which keeps the issue loop to the MMAs themselves.
        const uint64_t kdesc0 = tc::sw128_desc(kvb, 16u, 1024u);
        int g = 0, c = 0, ku = 0;  // ring steps, this tile's steps, this tile's items
        bool ok = true;
        for (;;) {
            ScoredSlot sl;
            ok = take(u, ku, sl);
            if (!ok || sl.end) break;
            const ScoredItem it = sl.it;
            const int x = ku & 1;
            const uint32_t qpar = (uint32_t)(ku >> 1) & 1u;
            ++ku;
            if (lane == 0) mbar_arrive(q_free(u, x));  // done with the slot
            if (u >= it.tiles) {
                // no rows in this tile: release each K stage as it lands
                for (int j = 0; ok && j < it.nch; ++j, ++g) {
                    const int st = g % C::kStages;
                    ok = mbar_wait_bounded(k_full(st), (uint32_t)(g / C::kStages) & 1u, kWaitLimit);
                    if (ok && lane == 0) mbar_arrive(k_empty(st));
                    __syncwarp();
                }
                if (!ok) break;
                continue;
            }
            ok = mbar_wait_bounded(q_full(u, x), qpar, kWaitLimit);
            const uint64_t qdesc = tc::sw128_desc(qtile(x, u), 16u, 1024u);
            for (int j = 0; ok && j < it.nch; ++j, ++g, ++c) {
                const int st = g % C::kStages;
                const int b = c % kSB;
                ok = mbar_wait_bounded(k_full(st), (uint32_t)(g / C::kStages) & 1u, kWaitLimit);
                // S/P[u][b] is free once the P V of this tile's step c - kSB has read P from it
                if (ok && c >= kSB) ok = mbar_wait_bounded(o_done(u, b), (uint32_t)((c / kSB) - 1) & 1u, kWaitLimit);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint64_t kdesc = tc::desc_add(kdesc0, (uint32_t)(st * C::kStageBytes));
                    const uint32_t sd = tbase + s_col(u, b);
#pragma unroll
                    for (int k = 0; k < C::kKS; ++k) {
                        tc::mma_f16_ss(sd, tc::desc_add(qdesc, (uint32_t)((k >> 2) * C::kQHalf + 32 * (k & 3))),
                                       tc::desc_add(kdesc, (uint32_t)((k >> 2) * C::kHalf + 32 * (k & 3))), idesc_s,
                                       k > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(s_full(u, b));
                    tc::mma_commit(k_empty(st));  // the K stage is free once every tile's S MMAs complete
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
        // every MMA issued by this thread has completed before TMEM is freed
        if (lane == 0) tc::mma_commit(drain_s(u));
        __syncwarp();
        mbar_wait_bounded(drain_s(u), 0u, kWaitLimit);
    } else if (warp == 3 || (MT == 2 && warp == 5)) {
        // ------------------------------------------------------------ O += P V issuer of tile u
        // Threads of their own: issuing S MMAs may block while the tensor pipe is
        // busy, and must not hold back a P V whose P is ready.  An item's first
        // P V overwrites O: its P is published after the softmax warps have read
        // the previous item's O out in their epilogue.
        const int u = warp == 3 ? 0 : 1;
        constexpr uint32_t idesc_o = tc::f16_idesc(kBf16, true, C::kM, D);
        const uint64_t vdesc0 = tc::sw128_desc(kvb + (uint32_t)C::kTile, (uint32_t)C::kHalf, 1024u);
        const uint32_t od = tbase + o_col(u);
        int g = 0, c = 0, ku = 0;
        bool ok = true;
        for (;;) {
            ScoredSlot sl;
            ok = take(u, ku, sl);
            if (!ok || sl.end) break;
            const ScoredItem it = sl.it;
            if (lane == 0) mbar_arrive(q_free(u, ku & 1));  // done with the slot
            ++ku;
            if (u >= it.tiles) {
                // no rows in this tile: release each V stage as it lands
                for (int j = 0; ok && j < it.nch; ++j, ++g) {
                    const int st = g % C::kStages;
                    ok = mbar_wait_bounded(v_full(st), (uint32_t)(g / C::kStages) & 1u, kWaitLimit);
                    if (ok && lane == 0) mbar_arrive(v_empty(st));
                    __syncwarp();
                }
                if (!ok) break;
                continue;
            }
            for (int j = 0; ok && j < it.nch; ++j, ++g, ++c) {
                const int b = c % kSB;
                const int st = g % C::kStages;
                ok = mbar_wait_bounded(v_full(st), (uint32_t)(g / C::kStages) & 1u, kWaitLimit);
                if (__builtin_expect((it.s & kHoles) != 0, 0) && __all_sync(0xffffffffu, ok)) {
                    // V rows between the rows' ranges hold anything, and a weight of 0 does not keep NaN out: the keys
                    // that no token of the item (of either tile) sees are zeroed, by each tile's issuer for itself (the same
                    // zeros). Ranges are read again and the item from its slot, the tile's until its softmax is done,
                    // so that the other items' steps keep none of it in registers.
                    const ScoredItem &of = slot(u, (ku - 1) & 1).it;
                    const int k0 = (of.lo / C::kN + j) * C::kN;
                    uint32_t any[C::kN / 32] = {};
                    for (int t = of.r0 / G + lane; t < min(of.n, (of.r0 + C::kM * MT) / G); t += 32) {
                        const int2 k = row_range(a, of.qs + t, of.len - of.n + t, of.len);
#pragma unroll
                        for (int w = 0; w < C::kN / 32; ++w)
                            any[w] |= bits_below(k.y - k0 - 32 * w) & ~bits_below(k.x - k0 - 32 * w);
                    }
#pragma unroll
                    for (int w = 0; w < C::kN / 32; ++w)
                        if (!(__reduce_or_sync(0xffffffffu, any[w]) >> lane & 1u))
                            zero_v_row(kvb + (uint32_t)(st * C::kStageBytes + C::kTile + (32 * w + lane) * 128));
                    tc::fence_async_smem();
                    __syncwarp();
                }
                // tile 0's softmax zeroes the V rows that must not contribute; tile 0's own
                // P V is issued after that (its P is published after the zeroing)
                if (ok && u > 0) ok = mbar_wait_bounded(v_zeroed(g), (uint32_t)(g / C::kMasks) & 1u, kWaitLimit);
                if (ok) ok = mbar_wait_bounded(p_full(u, b), (uint32_t)(c / kSB) & 1u, kWaitLimit);
                if (!ok) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint64_t vdesc = tc::desc_add(vdesc0, (uint32_t)(st * C::kStageBytes));
                    const uint32_t pa0 = tbase + s_col(u, b);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
#pragma unroll
                        for (int k = 0; k < C::kN / 16; ++k)
                            tc::mma_f16_ts(od, pa0 + (uint32_t)((C::kN / 2) * part + 8 * k), tc::desc_add(vdesc, 2048u * k),
                                           idesc_o, (j > 0 || part > 0 || k > 0) ? 1u : 0u);
                    }
                    tc::mma_commit(o_done(u, b));
                    tc::mma_commit(v_empty(st));
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
        if (lane == 0) tc::mma_commit(drain_p(u));
        __syncwarp();
        mbar_wait_bounded(drain_p(u), 0u, kWaitLimit);
    }
    } else {
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;\n" ::: "memory");
        // ------------------------------------------------------------ softmax (one row per thread)
        const int u = (warp - C::kSoftWarp0) / 4;  // tile of this warpgroup
        const int wq = warp & 3;                 // TMEM lanes 32 * wq .. 32 * wq + 31
        const int r = 32 * wq + lane;            // row within the tile
        const float sl = a.scale * kLog2e;
        // a bias in the units of the logits below (raw, or log2 with a scale that is not positive)
        const float slope_units = kMode == kGeneral && !(sl > 0.f) ? 1.f : 1.f / sl;
        // kCapFixed: capped logits lie within c = cap log2(e) <= 80 of 0, so with bf16 weights (the
        // exponents of fp32) a constant, max(0, c - 48), does for the maximum: weights and their
        // low parts stay normal numbers (2^-121 and above), and sums of 2^22 weights of at most 2^48
        // leave values up to 2^58 room: no maximum, no rescaling.  A bias has no such bound.
        const float fixed_max = fmaxf(0.f, a.softcap * kLog2e - 48.f);
        // The maximum may lag by kLag octaves before O is rescaled, so f16 weights are lifted by as much less
        // (kWeightLift): they keep down to 2^-32 of the largest. (A lag of 4 keeps 2^-36, and took 378 us instead of 360 on
        // 16 x 512 capped f16 chunks, 6 took 371.)
        constexpr float kLag = 8.f, kLift = kBf16 ? 0.f : kWeightLift<T> - kLag;
        constexpr bool kCap = kMode == kCapFixed || kMode == kCapMax;
        constexpr bool kSlopes = kMode == kBias || kMode == kGeneral;
        const CapFit fit(a.softcap > 0.f ? a.scale / a.softcap : 0.f);
        static_assert(kMode != kCapFixed || kBf16, "f16 weights need the maximum");
        const uint32_t tl = tbase + ((uint32_t)(wq * 32) << 16);
        int g = 0, c = 0, ku = 0;
        bool ok = true;
        for (;;) {
            ScoredSlot item;
            ok = take(u, ku, item);
            if (!ok || item.end) {
                // A warp whose wait ran out joins the others' next decision all the same: each warp goes through one
                // barrier for every item with rows here, and through one on its way out.
                warpgroup_all(1 + u, false);
                break;
            }
            const ScoredItem it = item.it;
            const int x = ku & 1;
            ++ku;
            if (u >= it.tiles) {
                // no rows in this tile: only the ring's step count moves on
                g += it.nch;
                __syncwarp();
                if (lane == 0) mbar_arrive(q_free(u, x));
                continue;
            }
            const int n = it.n, nch = it.nch;
            const int R = it.r0 + C::kM * u + r;
            const int t = R / G;
            const int pos = it.len - n + t;
            const int2 range = t < n ? row_range(a, it.qs + t, pos, it.len) : make_int2(0, 0);
            const float slope = kSlopes && a.slopes ? a.slopes[it.kvh * G + R % G] * kLog2e * slope_units : 0.f;
            const int k_first = it.lo / C::kN * C::kN;
            float m_used = kMode == kCapFixed ? fixed_max : -INFINITY, l = 0.f;
            for (int j = 0; j < nch; ++j, ++g, ++c) {
                const int b = c % kSB;
                const int st = g % C::kStages;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(s_full(u, b), (uint32_t)(c / kSB) & 1u, kWaitLimit));
                if (!ok) break;
                tc::fence_after_sync();
                uint32_t sv[C::kN / 32][32];
#pragma unroll
                for (int q = 0; q < C::kN / 32; ++q) tc::tmem_ld32(tl + s_col(u, b) + 32u * q, sv[q]);
                tc::tmem_wait_ld();
                const int mask = masks[g % C::kMasks];
                const int k0 = k_first + j * C::kN;  // first key of this step
                const int vb = range.x - k0, ve = range.y - k0;  // this row's keys of the step: vb <= cc < ve
                float f[C::kN];
#pragma unroll
                for (int cc = 0; cc < C::kN; ++cc) f[cc] = __uint_as_float(sv[cc >> 5][cc & 31]);
                // the step's keys that this row sees, a bit each (comparing positions key by key took ragged
                // prompts with a prefix mask, D 64, from 61 us to 65)
                uint32_t see[C::kN / 32];
#pragma unroll
                for (int w = 0; w < C::kN / 32; ++w) {
                    see[w] = bits_below(ve - 32 * w) & ~bits_below(vb - 32 * w) &
                             ((mask >> (2 * w) & 1 ? 0xffffu : 0u) | (mask >> (2 * w + 1) & 1 ? 0xffff0000u : 0u));
                }
                auto seen = [&](int cc) { return (see[cc >> 5] >> (cc & 31) & 1u) != 0u; };
                // raw units (the positive scale is folded into the exponent's FFMA), or log2 units here
                float mul = sl;
                if (kMode == kGeneral && !(sl > 0.f)) {
                    const ScoreCap score(a);
#pragma unroll
                    for (int cc = 0; cc < C::kN; ++cc) f[cc] = score(f[cc]);
                    mul = 1.f;
                } else if (kCap || (kMode == kGeneral && a.softcap > 0.f)) {
                    float am[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int cc = 0; cc < C::kN; cc += 2) am[cc >> 1 & 3] = max3(am[cc >> 1 & 3], fabsf(f[cc]), fabsf(f[cc + 1]));
                    float most = fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3]));
                    if (__all_sync(0xffffffffu, most <= fit.near)) {
                        cap_near(f, fit);
                    } else {
                        // which form a warp takes must not depend on what masked keys hold (asked only
                        // here: zeroing their logits in every step that has some took 350 us against 334)
                        most = 0.f;
#pragma unroll
                        for (int cc = 0; cc < C::kN; ++cc) most = fmaxf(most, seen(cc) ? fabsf(f[cc]) : 0.f);
                        cap_in_place(f, fit, most);
                    }
                }
                // bias: -slope |pos - key| = -slope (pos - k0) + slope cc where no key of the step lies
                // past pos (any step but the last of a prefix): the first part goes into the exponent's FFMA
                float shift = 0.f;
                if (kSlopes) {
                    const float d0 = (float)(pos - k0);
                    if (__all_sync(0xffffffffu, d0 >= (float)(C::kN - 1) || range.y <= pos + 1)) {
                        shift = -slope * d0;
#pragma unroll
                        for (int cc = 0; cc < C::kN; ++cc) f[cc] = fmaf(slope, (float)cc, f[cc]);  // an immediate each
                    } else {
#pragma unroll
                        for (int cc = 0; cc < C::kN; ++cc) f[cc] = fmaf(-slope, fabsf(d0 - (float)cc), f[cc]);
                    }
                }
                // every key of the step loaded and seen by all of the warp's rows
                const bool whole = __all_sync(0xffffffffu, vb <= 0 && ve >= C::kN) && mask == (1 << C::kBoxes) - 1;
                if (!whole) {
#pragma unroll
                    for (int cc = 0; cc < C::kN; ++cc)
                        if (!seen(cc)) f[cc] = -INFINITY;
                }
                // row maximum as 8 independent chains (a single 64-long chain of
                // dependent max operations would sit on the critical path)
                bool need = false;
                float alpha = 1.f;
                if (kMode != kCapFixed) {
                    float mx[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx[i] = f[i];
#pragma unroll
                    for (int cc = 8; cc < C::kN; ++cc) mx[cc & 7] = fmaxf(mx[cc & 7], f[cc]);
                    const float mr = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                           fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                    const float mc = (mr + shift) * mul - kLift;  // -inf when nothing is visible
                    need = mc > m_used + kLag;
                    alpha = (need && j > 0) ? ex2(m_used - mc) : 1.f;
                    if (need) m_used = mc;
                }
                const float mu = m_used == -INFINITY ? 0.f : m_used;
                // P = exp2(x - m) split into P_hi + P_lo, in registers before waiting,
                // two keys per packed f32x2 operation; the row sum in 4 pair accumulators
                uint32_t hw[C::kN / 2], lw[C::kN / 2];
                uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
                const uint64_t mul2 = tc::f2(mul, mul), nmu2 = tc::f2(shift * mul - mu, shift * mul - mu);
#pragma unroll
                for (int v = 0; v < C::kN / 2; ++v) {
                    const float2 xa = tc::f2split(tc::fma2(tc::f2(f[2 * v], f[2 * v + 1]), mul2, nmu2));
                    const float p0 = ex2(xa.x), p1 = ex2(xa.y);
                    const uint64_t pp = tc::f2(p0, p1);
                    ls[v & 3] = tc::add2(ls[v & 3], pp);
                    hw[v] = M::pack(p0, p1);
                    const float2 hf = M::unpack(hw[v]);
                    const float2 d = tc::f2split(tc::sub2(pp, tc::f2(hf.x, hf.y)));
                    lw[v] = M::pack(d.x, d.y);
                }
                const float2 s01 = tc::f2split(tc::add2(ls[0], ls[1])), s23 = tc::f2split(tc::add2(ls[2], ls[3]));
                l = l * alpha + ((s01.x + s01.y) + (s23.x + s23.y));
                // O may be rescaled only once the P V of step j - 1 has landed in it
                const bool rescale = j > 0 && __any_sync(0xffffffffu, need);
                if (rescale) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(o_done(u, (c - 1) % kSB),
                                                                    (uint32_t)((c - 1) / kSB) & 1u, kWaitLimit));
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {
                        uint32_t ov[16];
                        tc::tmem_ld16(tl + o_col(u) + 16u * q, ov);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tc::tmem_st16(tl + o_col(u) + 16u * q, ov);
                    }
                    tc::tmem_wait_st();
                }
                // P into TMEM over this step's S (already read): P_hi, then P_lo
                if constexpr (C::kN == 64) {
                    tc::tmem_st32(tl + s_col(u, b), hw);
                    tc::tmem_st32(tl + s_col(u, b) + 32u, lw);
                } else {
                    tc::tmem_st16(tl + s_col(u, b), hw);
                    tc::tmem_st16(tl + s_col(u, b) + 16u, lw);
                }
                tc::tmem_wait_st();
                // V rows of keys that were not loaded or lie outside the item's span hold
                // anything: tile 0's warpgroup zeroes them (row r < kN of this step's
                // V, whole 128-byte rows) before it publishes its P and v_zeroed, which
                // the other tile's P V issuer waits for.
                if (u == 0 && (k0 < it.lo || k0 + C::kN > it.hi || mask != (1 << C::kBoxes) - 1)) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(v_full(st), (uint32_t)(g / C::kStages) & 1u, kWaitLimit));
                    if (!ok) break;
                    if (r < C::kN && (k0 + r < it.lo || k0 + r >= it.hi || !(mask >> (r >> 4) & 1))) {
                        zero_v_row(kvb + (uint32_t)(st * C::kStageBytes + C::kTile + r * 128));
                        tc::fence_async_smem();
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(p_full(u, b));
                    if (u == 0) mbar_arrive(v_zeroed(g));
                }
            }
            const int last = c - 1;  // this tile's last step of the item
            if (ok)
                ok = __all_sync(0xffffffffu,
                                mbar_wait_bounded(o_done(u, last % kSB), (uint32_t)(last / kSB) & 1u, kWaitLimit));
            // One decision for the warpgroup: every warp reaches this barrier (all
            // its waits above are bounded), so the epilogue's barriers below are
            // entered by all four warps or by none.
            ok = warpgroup_all(1 + u, ok);
            if (!ok) break;
            // ---- epilogue: out = O / l, staged through the item's query tile (its S
            // MMAs are complete, so it is free).
            tc::fence_after_sync();
            tc::fence_async_smem();
            const float inv = l != 0.f ? 1.f / l : 0.f;  // a row with an empty range: zeros
            const uint32_t qt = qtile(x, u);
            const bool full = it.r0 + C::kM * (u + 1) <= n * G;  // all 128 rows belong to the chunk
            if (a.out16) {
                // 16-bit output: the query tile's own layout (halves of 64 columns, rows of 128
                // bytes in (token, head) order, 128-byte swizzle)
#pragma unroll
                for (int sb = 0; sb < C::kSub; ++sb) {
                    const uint32_t row = qt + (uint32_t)(sb * C::kQHalf + r * 128);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t ov[32];
                        tc::tmem_ld32(tl + o_col(u) + (uint32_t)(64 * sb + 32 * q), ov);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = M::pack(__uint_as_float(ov[8 * i + 2 * e]) * inv,
                                               __uint_as_float(ov[8 * i + 2 * e + 1]) * inv);
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             row + ((uint32_t)((4 * q + i) ^ (r & 7)) << 4)),
                                         "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                                         : "memory");
                        }
                    }
                }
                if (full) {
                    const bool issuer = wq == 0 && lane == 0;
                    tc::fence_async_smem();
                    warpgroup_sync(1 + u);
                    if (issuer) {
                        const uint64_t spol = policy_evict_first();
#pragma unroll
                        for (int sb = 0; sb < C::kSub; ++sb)
                            tma_store_3d(&tmo, qt + (uint32_t)(sb * C::kQHalf), 64 * sb, it.kvh * G,
                                         it.qs + (it.r0 + C::kM * u) / G, spol);
                        bulk_wait_read<0>();
                    }
                    warpgroup_sync(1 + u);
                } else {
                    // rows past the chunk: each warp writes its own rows, 8 lanes per 128 bytes
                    __syncwarp();
                    const int lg = __ffs(G) - 1;
#pragma unroll
                    for (int i = 0; i < 8 * C::kSub; ++i) {
                        const int rr = 32 * wq + 4 * (i & 7) + (lane >> 3), sb = i >> 3, cc = lane & 7;
                        const int Rr = it.r0 + C::kM * u + rr, tr = Rr >> lg;  // G is a power of two
                        const uint4 v = lds128(qt + (uint32_t)(sb * C::kQHalf + rr * 128) + ((uint32_t)(cc ^ (rr & 7)) << 4));
                        if (tr < n)
                            __stcs(reinterpret_cast<uint4 *>(static_cast<T *>(a.out) +
                                                             ((size_t)(it.qs + tr) * a.Hq + it.kvh * G + (Rr & (G - 1))) * D +
                                                             64 * sb + 8 * cc),
                                   v);
                    }
                    __syncwarp();
                }
            } else if (full) {
                // A tile whose 128 rows all belong to the chunk: 32-column blocks, each
                // staged as one TMA box (rows in (token, head) order, 128-byte
                // swizzle) and stored by one thread while the warpgroup moves on;
                // consecutive blocks take turns in the query tile's 16 KB parts.
                constexpr int kParts = C::kQTile / 16384;  // 2 (D 128) or 1 (D 64)
                const bool issuer = wq == 0 && lane == 0;
                const uint64_t spol = policy_evict_first();
#pragma unroll
                for (int cb = 0; cb < D / 32; ++cb) {
                    const uint32_t half = qt + (uint32_t)((cb % kParts) * 16384);
                    if (cb >= kParts) {
                        if (issuer) bulk_wait_read<kParts - 1>();  // the store of block cb - kParts has read this part
                        warpgroup_sync(1 + u);
                    }
                    uint32_t ov[32];
                    tc::tmem_ld32(tl + o_col(u) + (uint32_t)(32 * cb), ov);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(half + (uint32_t)(r * 128) +
                                                                                      ((uint32_t)(i ^ (r & 7)) << 4)),
                                     "f"(__uint_as_float(ov[4 * i]) * inv), "f"(__uint_as_float(ov[4 * i + 1]) * inv),
                                     "f"(__uint_as_float(ov[4 * i + 2]) * inv), "f"(__uint_as_float(ov[4 * i + 3]) * inv)
                                     : "memory");
                    tc::fence_async_smem();
                    warpgroup_sync(1 + u);
                    if (issuer) tma_store_3d(&tmo, half, 32 * cb, it.kvh * G, it.qs + (it.r0 + C::kM * u) / G, spol);
                }
                if (issuer) bulk_wait_read<0>();
                warpgroup_sync(1 + u);
            } else {
                // A tile with rows past the chunk: each warp stages its 32 rows, W
                // columns at a time (rows of W floats, 16-byte chunks swizzled by row),
                // then writes whole rows of the chunk's tokens to global memory,
                // lanes_per_row lanes per row, instead of one 16-byte piece of 32
                // different rows per store.
                constexpr int W = D / 2;                       // columns per pass
                constexpr int kRowBytes = W * 4;               // 256 (D 128) or 128 (D 64)
                constexpr int kRowsPerPiece = 4096 / kRowBytes;  // rows in one 4 KB piece of the warp's Q slice
                constexpr int kLanesPerRow = kRowBytes / 16;
                constexpr int kRowsPerStore = 32 / kLanesPerRow;
                const int lg = __ffs(G) - 1;
                const int rbase = it.r0 + C::kM * u + 32 * wq;  // tile row of this warp's first row
                auto stage = [&](int rr, int cc) {  // staging address of 16-byte chunk cc of row rr
                    return qt + (uint32_t)((rr / kRowsPerPiece) * C::kQHalf + wq * 32 * 128) +
                           (uint32_t)((rr % kRowsPerPiece) * kRowBytes) + ((uint32_t)(cc ^ (rr & 7)) << 4);
                };
#pragma unroll
                for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
                    for (int q = 0; q < W / 32; ++q) {
                        uint32_t ov[32];
                        tc::tmem_ld32(tl + o_col(u) + (uint32_t)(pass * W + 32 * q), ov);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage(lane, 8 * q + i / 4)),
                                         "f"(__uint_as_float(ov[i]) * inv), "f"(__uint_as_float(ov[i + 1]) * inv),
                                         "f"(__uint_as_float(ov[i + 2]) * inv), "f"(__uint_as_float(ov[i + 3]) * inv)
                                         : "memory");
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32 / kRowsPerStore; ++i) {
                        const int rr = i * kRowsPerStore + lane / kLanesPerRow;  // row of this warp's 32
                        const int cc = lane % kLanesPerRow;
                        const int Rr = rbase + rr;
                        const int tr = Rr >> lg;  // G is a power of two
                        const float4 v = *reinterpret_cast<const float4 *>(smem_raw + (stage(rr, cc) - raw));
                        if (tr < n)
                            __stcs(reinterpret_cast<float4 *>(static_cast<float *>(a.out) + ((size_t)(it.qs + tr) * a.Hq + it.kvh * G +
                                                                       (Rr & (G - 1))) * D + pass * W + 4 * cc),
                                   v);
                    }
                    __syncwarp();
                }
            }
            // the query-tile set may be reloaded (async proxy) after these generic-proxy reads
            tc::fence_async_smem();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_free(u, x));
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
        if (wq == 0 && lane == 0) bulk_wait_all();  // this thread's output stores have completed
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, C::kTmemCols);
    }
}

template <typename T, int D, int MT, int kMode>
cudaError_t launch_scored_umma_t(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                 const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    using C = ScoredUmmaCfg<D, MT, kMode>;
    static std::atomic<int> sms_of[kMaxLaunchDevices];
    int sms = 0;
    cudaError_t e = per_device_value(sms_of, &sms, [](int dev, int *v) {
        cudaError_t r = cudaFuncSetAttribute(scored_umma_kernel<T, D, MT, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)C::kSmem);
        if (r != cudaSuccess) return r;
        if (C::kRegSplit) {
            // the split draws on the registers of the launch: it must have been built for exactly these
            cudaFuncAttributes at;
            r = cudaFuncGetAttributes(&at, scored_umma_kernel<T, D, MT, kMode>);
            if (r != cudaSuccess) return r;
            if (at.numRegs != 128) return cudaErrorInvalidConfiguration;
        }
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
    });
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.max_query_len * (a.Hq / a.Hkv);
    const long long groups = (rows + C::kM * MT - 1) / (C::kM * MT);  // tile groups per sequence, at most
    const long long work = groups * a.S * a.Hkv;                       // list entries x KV heads, at most
    if (work > 0x7fffffffLL) return cudaErrorInvalidValue;
    // persistent: one CTA per SM (the shared memory admits no second one)
    const long long ctas = work < sms ? work : sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas > 0 ? ctas : 1));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_umma_kernel<T, D, MT, kMode>, a, tmk, tmv, tmq, tmo);
}

// Two tiles per CTA once a sequence can fill them (chunk_umma_rows).
template <typename T, int kMode>
cudaError_t launch_scored_umma(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                               const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    if (a.D == 64)
        return a.umma_rows == 256 ? launch_scored_umma_t<T, 64, 2, kMode>(a, tmk, tmv, tmq, tmo, st)
                                  : launch_scored_umma_t<T, 64, 1, kMode>(a, tmk, tmv, tmq, tmo, st);
    if (a.D == 128)
        return a.umma_rows == 256 ? launch_scored_umma_t<T, 128, 2, kMode>(a, tmk, tmv, tmq, tmo, st)
                                  : launch_scored_umma_t<T, 128, 1, kMode>(a, tmk, tmv, tmq, tmo, st);
    return cudaErrorNotSupported;
}

}  // namespace pa
