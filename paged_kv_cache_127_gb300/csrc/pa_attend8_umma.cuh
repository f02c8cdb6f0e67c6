// pa_attend8_umma.cuh -- long chunks over the 8-bit cache (the formulas are in
// pa_attend8.cuh) on the 5th-generation tensor cores: tcgen05.mma with operands in
// shared memory and the accumulators in tensor memory (TMEM).
//
// Work: an item is (MT 128-row tiles, KV head, sequence), row r = token r / G, head r % G; its CTA walks the keys
// that some of its rows see in steps of 64.  Persistent CTAs, one per SM, claim items from a longest-first list; or, where
// items are few and long, all items' steps stand in one line of which each CTA takes an equal stretch, pieces of items leave
// their (m, l, O) in the workspace, and a second launch joins them.  (The line for all calls: 356 us instead of 221 for
// 16 x 512 tokens, as each CTA then works on keys of its own instead of all on the same few sequences'.)  Warps:
//   0, 1       send for tile 0's and tile 1's queries (TMA) and issue  S_u = Q_u K^T  (M 128, N 64, K = D)
//   2, 3       issue their  O_u += P_u V    (M 128, N = D, K = 64), P from TMEM
//   4 .. 11    converters, a warpgroup for K and one for V, each warp with one 16-key box of every step: it loads its
//              box's codes a step ahead, turns them into 16-bit floats (K into the queries' type, V into f16; both
//              exact) and stores them as the swizzled operands; K's also publish the box's scales, and warp 4
//              publishes the items.
//   12 ..      one softmax warpgroup per tile, one thread per row
// Converting once per step serves both tiles, and the codes' 16-bit form never leaves the SM.  The alternative, e4m3
// operands with Q and P split in two terms each, would need as many products, and the split of P in the softmax
// costs it more instructions than the whole conversion takes here.
//
// The softmax applies scales per 16-key box: the box's largest score times ks (with log2 vs added) enters the row's
// maximum, the exponent's multiply-add carries ks and log2 vs, and the box's sum of weights 1 / vs.  The running
// maximum moves only when a row's new one is 2^8 larger, as in the kernel for 16-bit caches.
//
// Synchronisation is by mbarriers, every wait bounded: on a timeout the kernel sets PA_DEVERR_TIMEOUT, waits
// (bounded) for the MMAs and copies it issued, frees its TMEM and returns.  (A softmax warpgroup's own barriers have
// no limit: each of its warps goes through as many of them, whatever it gave up on.)
#pragma once

#include <cuda.h>

#include <cmath>
#include <type_traits>

#include "pa_attend8.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

template <int D, int MT>
struct Umma8Cfg {
    static constexpr int kM = 128;                         // rows per tile (TMEM lanes)
    static constexpr int kN = 64;                          // keys per step
    static constexpr int kSB = 2;                          // S/P buffers per tile
    static constexpr int kBoxes = kN / 16;                 // 16-key boxes of a step
    static constexpr int kSub = D / 64;                    // 128-byte halves of an operand row
    static constexpr int kKS = D / 16;                     // k-steps of S = Q K^T
    static constexpr int kStages = 3;
    static constexpr int kThreads = 32 * (12 + 4 * MT);
    // two tiles: 640 threads are launched at 96 registers; the issuers keep 40, the converters 88, the softmax gets 128
    // (4 x 40 + 8 x 88 + 8 x 128 < 20 x 96)
    static constexpr bool kRegSplit = MT == 2;
    static constexpr int kHalf = kN * 128;                 // one half of K (or V) of a step
    static constexpr int kTile = kSub * kHalf;             // K (or V) of a step
    static constexpr int kStageBytes = 2 * kTile;
    static constexpr int kQHalf = kM * 128;
    static constexpr int kQTile = kSub * kQHalf;
    // scales of the last kNotes steps.  Those of step g + 1 are written once step g is converted, so once S of
    // g - kStages is done, so once tile 0's P V of kSB steps before that is, whose V came when both tiles' P V had
    // released that of kStages before: every tile has read what lies 2 kStages + kSB steps back from g
    static constexpr int kNotes = 16;
    static constexpr int kNoteBytes = 4 * 4 * kBoxes;      // per box: ck, lv, 1 / vs, 1 or 0 (not there)
    static constexpr size_t kKVOff = (size_t)MT * kQTile;
    static constexpr int kOutBytes = 32 * 256;             // of a softmax warp: its rows on their way out, 256 bytes at a time
    static constexpr size_t kOutOff = kKVOff + (size_t)kStages * kStageBytes;
    static constexpr size_t kNoteOff = kOutOff + (size_t)4 * MT * kOutBytes;
    static constexpr size_t kItemOff = kNoteOff + (size_t)kNotes * kNoteBytes;   // per tile two items of 16 ints
    static constexpr size_t kBarOff = kItemOff + (size_t)MT * 2 * 64;
    // k_full, k_empty, v_full, v_empty [kStages] | per tile: s_full, p_full, o_done [kSB],
    // item_free [2], item_ready [2], q_full, q_done, drain_s, drain_p
    static constexpr int kTileBars = 3 * kSB + 8;
    static constexpr int kNumBars = 4 * kStages + MT * kTileBars;
    static constexpr size_t kSlotOff = kBarOff + 8 * kNumBars;
    static constexpr size_t kSmem = kSlotOff + 16 + 1024;  // + alignment slack
    static constexpr uint32_t kTmemCols = 256 * MT;
    static constexpr uint32_t kOCol = 128 * MT;            // S[u][b] at 128 u + kN b; O[u] at kOCol + D u; P over its S
    static_assert(2 * kStages + kSB + 1 <= kNotes, "a note must outlive its readers");
    static_assert(kOCol + MT * D <= kTmemCols, "TMEM budget");
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// One work item, or a piece of one, as the converters publish it to a tile's roles; end: no more items.
struct Item8 {
    int s, kvh, r0, qs, n, len, tiles, v0, count, ns, gap, lo, hi, part, end;   // its steps v0 .. v0 + count - 1; part -1: the whole item
};
static_assert(sizeof(Item8) <= 64, "an item's share of shared memory");

template <typename C>
__device__ __forceinline__ bool umma_item8(const Attend8Args &a, int s, int group, int kvh, Item8 &it) {
    const int G = a.Hq / a.Hkv, MT = a.tiles;
    const Seq8 q = seq_of(a, s, false);
    it.s = s;
    it.kvh = kvh;
    it.r0 = group * C::kM * MT;
    it.v0 = 0;
    it.part = -1;
    it.qs = q.q0;
    it.n = q.n;
    it.len = q.len;
    it.tiles = min(MT, (q.n * G - it.r0 + C::kM - 1) / C::kM);
    const Span8 span = span_of(a, q, it.r0);
    it.hi = span.hi;
    it.lo = span.lo;
    const Steps8 st = span.st;
    it.ns = st.ns;
    it.gap = st.gap;
    it.count = st.count;
    return q.n * G > it.r0;
}

// Bits 0 .. x - 1 of a word (none for x <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int x) { return x >= 32 ? ~0u : (1u << max(x, 0)) - 1u; }

// 16 codes as 16-bit floats, for K in the queries' type.
template <typename T>
__device__ __forceinline__ void widen16(const uint4 &w, uint4 &x, uint4 &y) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = f16_of_codes(i & 1 ? in[i >> 1] >> 16 : in[i >> 1] & 0xffffu);
        if constexpr (std::is_same<T, __half>::value) {
            out[i] = h;
        } else {
            const float2 f = Mma16<__half>::unpack(h);
            out[i] = Mma16<T>::pack(f.x, f.y);
        }
    }
    x = make_uint4(out[0], out[1], out[2], out[3]);
    y = make_uint4(out[4], out[5], out[6], out[7]);
}

__device__ __forceinline__ void sts128(uint32_t at, const uint4 &x) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
// 16 codes, or zeros where there are none: the load is predicated, so that nothing waits for it before its use.
// (Not by the read-only path: this grid may start while the launch before it, a write into the cache, is still running.)
__device__ __forceinline__ void ldg_codes(uint4 &v, const uint8_t *p, bool want) {
    v = make_uint4(0, 0, 0, 0);
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"((uint32_t)want));
}
__device__ __forceinline__ float4 lds_f4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ bool group_all(int id, bool pred) {   // barrier over a warpgroup
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(id)
        : "memory");
    return r != 0;
}

// The ring's stage and phase follow the count g of steps so far, the S/P buffers and their phases the count c of the
// tile's own steps, the item slots and query-tile sets the count of items.
template <typename T, int D, int MT, bool kLine>
__global__ void __launch_bounds__(Umma8Cfg<D, MT>::kThreads, 1)
    attend8_umma_kernel(const Attend8Args a, const __grid_constant__ CUtensorMap tmq) {
    using C = Umma8Cfg<D, MT>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kSB = C::kSB;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *basep = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv;

    const uint32_t kvb = base + (uint32_t)C::kKVOff, bars = base + (uint32_t)C::kBarOff;
    auto k_full = [&](int i) { return bars + 8u * (uint32_t)i; };
    auto k_empty = [&](int i) { return bars + 8u * (uint32_t)(C::kStages + i); };
    auto v_full = [&](int i) { return bars + 8u * (uint32_t)(2 * C::kStages + i); };
    auto v_empty = [&](int i) { return bars + 8u * (uint32_t)(3 * C::kStages + i); };
    auto tbar = [&](int u, int i) { return bars + 8u * (uint32_t)(4 * C::kStages + u * C::kTileBars + i); };
    auto s_full = [&](int u, int b) { return tbar(u, b); };
    auto p_full = [&](int u, int b) { return tbar(u, kSB + b); };
    auto o_done = [&](int u, int b) { return tbar(u, 2 * kSB + b); };  // P V done: O is up to date, S/P[u][b] is free
    auto item_free = [&](int u, int x) { return tbar(u, 3 * kSB + x); };
    auto item_ready = [&](int u, int x) { return tbar(u, 3 * kSB + 2 + x); };
    auto q_full = [&](int u) { return tbar(u, 3 * kSB + 4); };
    auto q_done = [&](int u) { return tbar(u, 3 * kSB + 5); };   // the S MMAs of an item are complete
    auto drain_s = [&](int u) { return tbar(u, 3 * kSB + 6); };
    auto drain_p = [&](int u) { return tbar(u, 3 * kSB + 7); };
    Item8 *slots = reinterpret_cast<Item8 *>(basep + C::kItemOff);
    auto slot = [&](int u, int x) -> Item8 & { return *reinterpret_cast<Item8 *>(reinterpret_cast<unsigned char *>(slots) + 64 * (2 * u + x)); };
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kWaitLimit)); };
    auto take = [&](int u, int k, Item8 &out) {   // tile u's k-th item; false on a timeout
        const bool got = wait(item_ready(u, k & 1), (uint32_t)(k >> 1) & 1u);
        if (got) out = slot(u, k & 1);
        __syncwarp();  // every lane has read it before one of them frees the slot
        return got;
    };
    auto qtile = [&](int u) { return base + (uint32_t)(u * C::kQTile); };
    auto s_col = [&](int u, int b) { return (uint32_t)(128 * u + C::kN * b); };
    auto o_col = [&](int u) { return C::kOCol + (uint32_t)(D * u); };
    auto note = [&](int g) { return base + (uint32_t)(C::kNoteOff + (size_t)(g % C::kNotes) * C::kNoteBytes); };
    uint32_t *tslot = reinterpret_cast<uint32_t *>(basep + C::kSlotOff);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(k_full(i), 4);    // the converters
            mbar_init(k_empty(i), MT);  // one arrival per tile's S issuer (a commit, or a plain one without rows)
            mbar_init(v_full(i), 4);
            mbar_init(v_empty(i), MT);  // likewise from each tile's P V issuer
        }
        for (int u = 0; u < MT; ++u) {
            for (int b = 0; b < kSB; ++b) {
                mbar_init(s_full(u, b), 1);
                mbar_init(p_full(u, b), 4);
                mbar_init(o_done(u, b), 1);
            }
            for (int x = 0; x < 2; ++x) {
                mbar_init(item_free(u, x), 4 + 2);  // the softmax warps, and both issuers once they have read it
                mbar_init(item_ready(u, x), 1);
            }
            mbar_init(q_full(u), 1);
            mbar_init(q_done(u), 1);
            mbar_init(drain_s(u), 1);
            mbar_init(drain_p(u), 1);
        }
        fence_mbar_init();
        prefetch_tmap(&tmq);
    }
    if (warp == 0) tc::tmem_alloc(smem_addr(tslot), C::kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    griddep_wait();  // the plan's list, longest first
    const int nwork = kLine ? 0 : max(0, a.hdr[0]) * a.Hkv;

    // The converters of K or of V: warp w of the group has box w of every step.
    auto convert = [&](auto of_v) {
        constexpr bool kV = decltype(of_v)::value;
        constexpr int kLanes = D / 16;                 // lanes of a key's row, 16 codes each
        constexpr int kPass = 32 / kLanes;             // rows of a pass
        constexpr int kP = 16 / kPass;                 // passes: 4 (D 128) or 2
        const int box = warp & 3, row = lane / kLanes, ch = lane % kLanes;
        const int lb = __ffs(a.B) - 1;
        const bool first = !kV && box == 0;            // claims the items
        // a row's two 16-byte chunks of its swizzled operand; the second half's lanes store theirs in the other
        // order, which keeps a store free of bank conflicts
        const bool flip = (ch & 4) != 0;
        const uint8_t *cache = kV ? a.v_cache : a.k_cache;
        auto full = [&](int i) { return kV ? v_full(i) : k_full(i); };
        auto empty = [&](int i) { return kV ? v_empty(i) : k_empty(i); };
        const uint32_t ring = kvb + (kV ? (uint32_t)C::kTile : 0u) + (uint32_t)((ch >> 2) * C::kHalf + (16 * box + row) * 128);
        int g = 0, k = 0, j = 0, count = 0;            // ring steps, items, the step to fetch next and its item's
        int next_w = blockIdx.x;                       // a CTA's first item needs no claim
        int4 at_line = make_int4(0, 0, 0, 0);          // (entry, KV head, step, steps left)
        if constexpr (kLine) at_line = a.starts[blockIdx.x];
        Item8 it;
        bool ok = true;
        // per lane, for the item's steps 32 n + lane: where the box's codes are (null: no row sees them, or the block
        // is none), the note of the box (K), and which of its keys some row sees (V)
        const uint8_t *src = nullptr;
        float4 box_note = make_float4(1.f, 0.f, 1.f, 0.f);
        int seen = 0;                                  // bits: keys of the box
        // the next item; false when there is none (or on a timeout)
        auto next_item = [&]() {
            if (first) {
                const bool have = kLine ? at_line.w > 0 : next_w < nwork;
                it.end = !have;
                if (!kLine && have) {
                    const int4 e = a.list[next_w / a.Hkv];   // (sequence, tile group, -, -)
                    umma_item8<C>(a, e.x, e.y, next_w % a.Hkv, it);
                } else if (have) {
                    for (;; ++at_line.x) {
                        const bool there = umma_item8<C>(a, at_line.x / a.groups, at_line.x % a.groups, at_line.y, it);
                        if (there || at_line.x >= a.S * a.groups - 1) break;
                    }
                    const int all = it.count, n = min(at_line.w, all - at_line.z);
                    it.v0 = at_line.z;
                    it.count = n;
                    it.part = n == all ? -1 : 2 * (int)blockIdx.x + (k > 0);
                    if (n < all && at_line.z == 0 && lane == 0)
                        a.notes[blockIdx.x] = make_int4(at_line.x, at_line.y, it.part, 1 + (all - n + a.hdr[1] - 1) / a.hdr[1]);
                    at_line.w -= n;
                    at_line.z = 0;
                    if (++at_line.y == a.Hkv) at_line.y = 0, ++at_line.x;
                }
                const int x = k & 1;
#pragma unroll 1
                for (int u = 0; ok && u < MT; ++u) {
                    if (k >= 2) ok = wait(item_free(u, x), (uint32_t)((k >> 1) - 1) & 1u);
                    if (ok && lane == 0) {
                        slot(u, x) = it;
                        mbar_arrive(item_ready(u, x));
                    }
                    __syncwarp();
                }
                if (!kLine && have) {
                    int w = 0;
                    if (lane == 0) w = (int)gridDim.x + atomicAdd(&a.hdr[1], 1);
                    next_w = __shfl_sync(0xffffffffu, w, 0);
                }
            } else {
                ok = take(0, k, it);  // tile 0 has rows in every item
            }
            ++k;
            j = 0;
            count = it.count;
            return ok && !it.end;
        };
        // The next step's codes on their way into `w`, and its note (K); false past the last item.  What an arrive
        // releases includes this warp's loads, so these are sent for behind one step's arrive and used before the next one's.
        uint4 w[kP];
        uint32_t keys = 0;                             // V: the box's keys that some row sees
        auto fetch = [&]() {
            if (j == count && !next_item()) return false;
            if ((j & 31) == 0) {
                const int v = (kLine ? it.v0 : 0) + j + lane, b0 = (v < it.ns ? v : v + it.gap) * C::kN + 16 * box;
                const bool want = j + lane < it.count && b0 < it.hi && (b0 + 15 >= it.lo || b0 < a.sinks);
                const int id = want ? a.block_tables[(size_t)it.s * a.max_blocks + (b0 >> lb)] : 0;
                const bool good = want && (unsigned)id < (unsigned)a.N;
                const size_t bh = (size_t)id * a.Hkv + it.kvh;
                src = good ? cache + (bh * a.B + (b0 & (a.B - 1))) * D : nullptr;
                if constexpr (kV) {
                    seen = good ? (int)(low_bits(it.hi - b0) & (~low_bits(it.lo - b0) | low_bits(a.sinks - b0)) & 0xffffu) : 0;
                } else {
                    float ks = 1.f, vs = 1.f;
                    if (good) {
                        ks = a.k_scales[bh];
                        vs = a.v_scales[bh];
                    } else if (want) {
                        set_error(a.err, PA_DEVERR_BAD_BLOCK);
                    }
                    box_note = make_float4(ks * a.scale * kLog2e8, lg2(vs), 1.f / vs, good ? 1.f : 0.f);
                }
            }
            const uint8_t *from = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), j & 31));
            if constexpr (kV) keys = __shfl_sync(0xffffffffu, seen, j & 31);
            else if (lane == (j & 31))
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(note(g) + 16 * box), "f"(box_note.x), "f"(box_note.y),
                             "f"(box_note.z), "f"(box_note.w)
                             : "memory");
            // a key that no row of the item sees may hold anything: its V counts as zeros
#pragma unroll
            for (int n = 0; n < kP; ++n) ldg_codes(w[n], from + n * 512 + lane * 16, kV ? (keys >> (row + kPass * n) & 1u) : from != nullptr);
            ++j;
            return true;
        };
#pragma unroll 1
        for (bool more = fetch(); more; more = fetch()) {
            const int st = g % C::kStages;
            if (g >= C::kStages) ok = wait(empty(st), (uint32_t)((g / C::kStages) - 1) & 1u);
            if (!ok) break;
#pragma unroll
            for (int n = 0; n < kP; ++n) {
                const int r = row + kPass * n;
                uint4 x, y;
                if constexpr (kV) widen16<__half>(w[n], x, y);
                else widen16<T>(w[n], x, y);
                const uint32_t at = ring + (uint32_t)(st * C::kStageBytes + kPass * n * 128), sw = (uint32_t)(r & 7);
                const uint32_t c0 = ((uint32_t)(2 * (ch & 3)) ^ sw) << 4, c1 = ((uint32_t)(2 * (ch & 3) + 1) ^ sw) << 4;
                sts128(at + (flip ? c1 : c0), flip ? y : x);
                sts128(at + (flip ? c0 : c1), flip ? x : y);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(st));
            ++g;
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
    };

    if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------ converters: K (warps 4-7), V (8-11)
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n" ::: "memory");
        if (warp < 8) convert(std::integral_constant<bool, false>());
        else convert(std::integral_constant<bool, true>());
    } else if (warp < 4) {
        // one instruction for all four warps of the warpgroup, as setmaxnreg asks
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n" ::: "memory");
        const int u = warp & 1;
        if (u < MT && warp < 2) {
            // -------------------------------------------------------- S = Q K^T issuer of tile u
            constexpr uint32_t idesc_s = tc::f16_idesc(kBf16, false, C::kM, C::kN);
            const uint64_t kdesc0 = tc::sw128_desc(kvb, 16u, 1024u);
            const uint64_t qpol = policy_evict_first();
            const uint64_t qdesc = tc::sw128_desc(qtile(u), 16u, 1024u);
            int g = 0, c = 0, k = 0, nq = 0;  // nq: items with rows in this tile
            bool ok = true;
            for (;;) {
                Item8 it;
                ok = take(u, k, it);
                if (!ok || it.end) break;
                if (lane == 0) mbar_arrive(item_free(u, k & 1));  // done with the slot
                ++k;
                if (u >= it.tiles) {
                    for (int j = 0; ok && j < it.count; ++j, ++g) {
                        const int st = g % C::kStages;
                        ok = wait(k_full(st), (uint32_t)(g / C::kStages) & 1u);
                        if (ok && lane == 0) mbar_arrive(k_empty(st));
                        __syncwarp();
                    }
                    if (!ok) break;
                    continue;
                }
                // the query tile, once the MMAs of the last one are complete: rows r0 + 128 u .., G heads of a token at
                // a time; rows of tokens past the chunk are never used
                if (nq > 0) ok = wait(q_done(u), (uint32_t)(nq - 1) & 1u);
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(q_full(u), (uint32_t)C::kQTile);
#pragma unroll
                    for (int sb = 0; sb < C::kSub; ++sb)
                        tma_load_3d(qtile(u) + (uint32_t)(sb * C::kQHalf), &tmq, sb * 64, it.kvh * G, it.qs + (it.r0 + C::kM * u) / G,
                                    q_full(u), qpol);
                }
                __syncwarp();
                if (ok) ok = wait(q_full(u), (uint32_t)nq & 1u);
                ++nq;
                for (int j = 0; ok && j < it.count; ++j, ++g, ++c) {
                    const int st = g % C::kStages, b = c % kSB;
                    ok = wait(k_full(st), (uint32_t)(g / C::kStages) & 1u);
                    if (ok && c >= kSB) ok = wait(o_done(u, b), (uint32_t)((c / kSB) - 1) & 1u);  // P V has read P[u][b]
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint64_t kdesc = tc::desc_add(kdesc0, (uint32_t)(st * C::kStageBytes));
                        const uint32_t sd = tbase + s_col(u, b);
#pragma unroll
                        for (int i = 0; i < C::kKS; ++i)
                            tc::mma_f16_ss(sd, tc::desc_add(qdesc, (uint32_t)((i >> 2) * C::kQHalf + 32 * (i & 3))),
                                           tc::desc_add(kdesc, (uint32_t)((i >> 2) * C::kHalf + 32 * (i & 3))), idesc_s, i > 0 ? 1u : 0u);
                        tc::mma_commit(s_full(u, b));
                        tc::mma_commit(k_empty(st));
                        if (j + 1 == it.count) tc::mma_commit(q_done(u));
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
        } else if (u < MT) {
            // -------------------------------------------------------- O += P V issuer of tile u
            constexpr uint32_t idesc_o = tc::f16_idesc(false, true, C::kM, D);
            const uint64_t vdesc0 = tc::sw128_desc(kvb + (uint32_t)C::kTile, (uint32_t)C::kHalf, 1024u);
            const uint32_t od = tbase + o_col(u);
            int g = 0, c = 0, k = 0;
            bool ok = true;
            for (;;) {
                Item8 it;
                ok = take(u, k, it);
                if (!ok || it.end) break;
                if (lane == 0) mbar_arrive(item_free(u, k & 1));
                ++k;
                if (u >= it.tiles) {
                    for (int j = 0; ok && j < it.count; ++j, ++g) {
                        const int st = g % C::kStages;
                        ok = wait(v_full(st), (uint32_t)(g / C::kStages) & 1u);
                        if (ok && lane == 0) mbar_arrive(v_empty(st));
                        __syncwarp();
                    }
                    if (!ok) break;
                    continue;
                }
                for (int j = 0; ok && j < it.count; ++j, ++g, ++c) {
                    const int b = c % kSB, st = g % C::kStages;
                    ok = wait(v_full(st), (uint32_t)(g / C::kStages) & 1u);
                    if (ok) ok = wait(p_full(u, b), (uint32_t)(c / kSB) & 1u);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint64_t vdesc = tc::desc_add(vdesc0, (uint32_t)(st * C::kStageBytes));
                        const uint32_t pa0 = tbase + s_col(u, b);
#pragma unroll
                        for (int i = 0; i < C::kN / 16; ++i)
                            tc::mma_f16_ts(od, pa0 + (uint32_t)(8 * i), tc::desc_add(vdesc, 2048u * i), idesc_o, (j > 0 || i > 0) ? 1u : 0u);
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
        // ------------------------------------------------------------ softmax (one row per thread)
        if constexpr (C::kRegSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;\n" ::: "memory");
        const int u = (warp - 12) / 4;
        const int wq = warp & 3;                 // TMEM lanes 32 wq ..
        const uint32_t tl = tbase + ((uint32_t)(wq * 32) << 16);
        int g = 0, c = 0, k = 0;
        bool ok = true;
        for (;;) {
            Item8 it;
            ok = take(u, k, it);
            if (!ok || it.end) {
                // A warp whose wait ran out joins the others' next decision all the same: each warp goes through one
                // barrier for every item with rows here, and through one on its way out.
                group_all(1 + u, false);
                break;
            }
            const int x = k & 1;
            ++k;
            if (u >= it.tiles) {
                g += it.count;
                __syncwarp();
                if (lane == 0) mbar_arrive(item_free(u, x));
                continue;
            }
            const int R = it.r0 + C::kM * u + 32 * wq + lane, t = R / G;
            const int pos = t < it.n ? it.len - it.n + t : it.len - 1;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < it.count; ++j, ++g, ++c) {
                const int b = c % kSB;
                ok = wait(s_full(u, b), (uint32_t)(c / kSB) & 1u);
                if (!ok) break;
                tc::fence_after_sync();
                uint32_t sv[2][32];
                tc::tmem_ld32(tl + s_col(u, b), sv[0]);
                tc::tmem_ld32(tl + s_col(u, b) + 32u, sv[1]);
                const uint32_t nt = note(g);
                const float4 n4[4] = {lds_f4(nt), lds_f4(nt + 16), lds_f4(nt + 32), lds_f4(nt + 48)};
                float ck[4] = {n4[0].x, n4[1].x, n4[2].x, n4[3].x}, lv[4] = {n4[0].y, n4[1].y, n4[2].y, n4[3].y};
                const float iv[4] = {n4[0].z, n4[1].z, n4[2].z, n4[3].z};
                const bool whole = fminf(fminf(n4[0].w, n4[1].w), fminf(n4[2].w, n4[3].w)) > 0.f;
                const int v = (kLine ? it.v0 : 0) + j, kb = (v < it.ns ? v : v + it.gap) * C::kN;
                const int lim = pos - kb;                                     // last visible key of the step
                const int from = a.window > 0 ? max(lim, -1) - a.window + 1 : 0;   // first one of the window
                tc::tmem_wait_ld();
                float f[C::kN];
#pragma unroll
                for (int i = 0; i < C::kN; ++i) f[i] = __uint_as_float(sv[i >> 5][i & 31]);
                const bool plain = fminf(fminf(ck[0], ck[1]), fminf(ck[2], ck[3])) >= 0x1p-120f;
                if (!(__all_sync(0xffffffffu, lim >= C::kN - 1 && (from <= 0 || kb + C::kN <= a.sinks)) && whole && plain)) {
                    // a step on the diagonal, on a window's border, over a block not loaded; a scale that is not positive
                    const int sk = a.window > 0 ? a.sinks - kb : 0;
                    uint32_t see[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        see[h] = low_bits(lim + 1 - 32 * h) & (~low_bits(from - 32 * h) | low_bits(sk - 32 * h));
                        see[h] &= (n4[2 * h].w > 0.f ? 0xffffu : 0u) | (n4[2 * h + 1].w > 0.f ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < C::kN; ++i) {
                        if (!plain) f[i] = fmaf(f[i], ck[i >> 4], lv[i >> 4]);
                        if (!(see[i >> 5] >> (i & 31) & 1u)) f[i] = -INFINITY;
                    }
                    if (!plain) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) ck[i] = 1.f, lv[i] = 0.f;
                    }
                }
                // the row's maximum: of each box's scores, then scaled
                float mc = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y = max3f(f[16 * q], f[16 * q + 1], f[16 * q + 2]), z = max3f(f[16 * q + 3], f[16 * q + 4], f[16 * q + 5]);
#pragma unroll
                    for (int i = 6; i < 14; i += 4) {
                        y = max3f(y, f[16 * q + i], f[16 * q + i + 1]);
                        z = max3f(z, f[16 * q + i + 2], f[16 * q + i + 3]);
                    }
                    y = max3f(y, f[16 * q + 14], f[16 * q + 15]);
                    mc = fmaxf(mc, fmaf(fmaxf(y, z), ck[q], lv[q]));
                }
                const bool need = mc > m + (8.f + kLift8);
                const float to = mc - kLift8;
                const float alpha = (need && j > 0) ? ex2(m - to) : 1.f;
                if (need) m = to;
                const float mu = m == -INFINITY ? 0.f : m;
                uint32_t pw[C::kN / 2];
                l *= alpha;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float nm = lv[q] - mu;
                    const uint64_t ck2 = tc::f2(ck[q], ck[q]), nm2 = tc::f2(nm, nm);
                    uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int v = 8 * q + i;
                        const float2 y = tc::f2split(tc::fma2(tc::f2(f[2 * v], f[2 * v + 1]), ck2, nm2));
                        const float p0 = ex2(y.x), p1 = ex2(y.y);
                        if (i & 1) s1 = tc::add2(s1, tc::f2(p0, p1));
                        else s0 = tc::add2(s0, tc::f2(p0, p1));
                        pw[v] = Mma16<__half>::pack(p0, p1);
                    }
                    const float2 s = tc::f2split(tc::add2(s0, s1));
                    l = fmaf(s.x + s.y, iv[q], l);
                }
                // O may be rescaled only once the P V of the step before has landed in it
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    ok = wait(o_done(u, (c - 1) % kSB), (uint32_t)((c - 1) / kSB) & 1u);
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
                tc::tmem_st32(tl + s_col(u, b), pw);   // P over the S just read
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(u, b));
            }
            const int last = c - 1;
            if (ok) ok = wait(o_done(u, last % kSB), (uint32_t)(last / kSB) & 1u);
            // one decision for the warpgroup
            ok = group_all(1 + u, ok);
            if (!ok) break;
            tc::fence_after_sync();
            const bool in_part = kLine && it.part >= 0;
            const float inv = in_part ? 1.f : l == 0.f ? 0.f : 1.f / l;
            float *part = a.parts + (size_t)(in_part ? it.part : 0) * (C::kM * MT) * (D + 2);
            if (in_part) *reinterpret_cast<float2 *>(part + (size_t)(C::kM * MT) * D + 2 * (C::kM * u + 32 * wq + lane)) = make_float2(m, l);
            // through shared memory, so that a store writes whole rows: 32 columns a turn into it, in 16-byte pieces swizzled by
            // row, then up to 256 bytes of each row out of it
            const uint32_t stage = base + (uint32_t)(C::kOutOff + (size_t)(warp - 12) * C::kOutBytes);
            const int lg = __ffs(G) - 1, R0 = it.r0 + C::kM * u + 32 * wq;   // this warp's first row; G is a power of two
            auto put = [&](int piece, const uint4 &v) { sts128(stage + (uint32_t)(lane * 256) + ((uint32_t)(piece ^ (lane & 7)) << 4), v); };
            auto flush = [&](int bytes, int at) {   // `bytes` of each row, to byte `at` of its head's output
                __syncwarp();
                const int per = bytes >> 4, each = 32 / per;        // lanes of a row, rows of a store
                const size_t row_bytes = (size_t)D * (a.out16 ? 2 : 4);
#pragma unroll 4
                for (int r = lane / per; r < 32; r += each) {
                    const int piece = lane % per, Rr = R0 + r, tr = Rr >> lg;
                    const uint4 v = lds128(stage + (uint32_t)(r * 256) + ((uint32_t)(piece ^ (r & 7)) << 4));
                    unsigned char *row = in_part ? reinterpret_cast<unsigned char *>(part + (size_t)(Rr - it.r0) * D)
                                                 : static_cast<unsigned char *>(a.out) + ((size_t)(it.qs + tr) * a.Hq + it.kvh * G + (Rr & (G - 1))) * row_bytes;
                    if (tr < it.n) *reinterpret_cast<uint4 *>(row + at + 16 * piece) = v;
                }
                __syncwarp();
            };
#pragma unroll
            for (int cb = 0; cb < D / 32; ++cb) {
                uint32_t ov[32];
                tc::tmem_ld32(tl + o_col(u) + (uint32_t)(32 * cb), ov);
                tc::tmem_wait_ld();
                if (a.out16 && !in_part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = Mma16<T>::pack(__uint_as_float(ov[8 * i + 2 * e]) * inv, __uint_as_float(ov[8 * i + 2 * e + 1]) * inv);
                        put(4 * cb + i, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                    if (cb == D / 32 - 1) flush(2 * D, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(__uint_as_float(ov[4 * i + e]) * inv);
                        put(8 * (cb & 1) + i, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                    if (cb & 1) flush(256, 256 * (cb >> 1));
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(item_free(u, x));
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, C::kTmemCols);
    }
}

// CTA (x, y): where CTA x of the line began an item that others went on with, rows 32 y .. of that item's parts joined,
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,   M = max m_i,
// a warp for four rows at a time, a lane D / 32 columns of each.
template <typename T, int D, int MT>
__global__ void __launch_bounds__(256) attend8_join_kernel(const Attend8Args a) {
    constexpr int kRows = 128 * MT, kPer = D / 32, kR = 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    griddep_wait();
    const int4 note = a.notes[blockIdx.x];   // (entry, KV head, the first part's slot, parts)
    // (parts past the last CTA's: none, as when the CTA gave up on a wait before it noted anything)
    if (note.w <= 0 || note.w > a.units - (int)blockIdx.x) return;
    const int G = a.Hq / a.Hkv, lg = __ffs(G) - 1, lane = threadIdx.x & 31;
    const Seq8 q = seq_of(a, note.x / a.groups, false);
    const int row0 = 32 * blockIdx.y + kR * (threadIdx.x >> 5), R0 = note.x % a.groups * kRows + row0;
    if (R0 >= q.n * G) return;
    auto part = [&](int i) { return a.parts + (size_t)(i == 0 ? note.z : 2 * ((int)blockIdx.x + i)) * kRows * (D + 2); };
    auto ml = [&](int i, int r) { return *reinterpret_cast<const float2 *>(part(i) + (size_t)kRows * D + 2 * (row0 + r)); };
    float M[kR], l[kR], o[kR][kPer];
#pragma unroll
    for (int r = 0; r < kR; ++r) M[r] = -INFINITY;
    for (int i = lane; i < note.w; i += 32)
#pragma unroll
        for (int r = 0; r < kR; ++r) M[r] = fmaxf(M[r], ml(i, r).x);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M[r] = fmaxf(M[r], __shfl_xor_sync(0xffffffffu, M[r], x));
        if (M[r] == -INFINITY) M[r] = 0.f;
        l[r] = 0.f;
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[r][x] = 0.f;
    }
#pragma unroll 4
    for (int i = 0; i < note.w; ++i) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const float2 y = ml(i, r);
            const float w = ex2(y.x - M[r]), *at = part(i) + (size_t)(row0 + r) * D + kPer * lane;
            l[r] = fmaf(w, y.y, l[r]);
#pragma unroll
            for (int x = 0; x < kPer; x += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(at + x);
                o[r][x] = fmaf(w, v.x, o[r][x]);
                o[r][x + 1] = fmaf(w, v.y, o[r][x + 1]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        const int R = R0 + r, t = R >> lg;
        if (t >= q.n) break;
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        const size_t at = ((size_t)(q.q0 + t) * a.Hq + note.y * G + (R & (G - 1))) * D + kPer * lane;
        if (a.out16) {
#pragma unroll
            for (int x = 0; x < kPer; x += 2) *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at + x) = Mma16<T>::pack(o[r][x] * inv, o[r][x + 1] * inv);
        } else {
#pragma unroll
            for (int x = 0; x < kPer; ++x) static_cast<float *>(a.out)[at + x] = o[r][x] * inv;
        }
    }
}

template <typename T, int D, int MT>
cudaError_t launch_umma8_t(const Attend8Args &a, const CUtensorMap &tmq, cudaStream_t st) {
    using C = Umma8Cfg<D, MT>;
    static std::atomic<int> sms_of[kMaxLaunchDevices];
    int sms = 0;
    cudaError_t e = per_device_value(sms_of, &sms, [](int dev, int *v) {
        cudaError_t r = cudaFuncSetAttribute(attend8_umma_kernel<T, D, MT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(attend8_umma_kernel<T, D, MT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (r != cudaSuccess) return r;
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
    });
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.max_query_len * (a.Hq / a.Hkv);
    const long long work = (rows + C::kM * MT - 1) / (C::kM * MT) * a.S * a.Hkv;
    if (work > 0x7fffffffLL) return cudaErrorInvalidValue;
    const long long ctas = a.units ? a.units : work < sms ? work : sms;
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
    if (!a.units) return cudaLaunchKernelEx(&cfg, attend8_umma_kernel<T, D, MT, false>, a, tmq);
    e = cudaLaunchKernelEx(&cfg, attend8_umma_kernel<T, D, MT, true>, a, tmq);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)a.units, 4u * MT);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attend8_join_kernel<T, D, MT>, a);
}

template <typename T>
cudaError_t dispatch_umma8(const Attend8Args &a, const CUtensorMap &tmq, cudaStream_t st) {
    if (a.D == 64) return a.tiles == 2 ? launch_umma8_t<T, 64, 2>(a, tmq, st) : launch_umma8_t<T, 64, 1>(a, tmq, st);
    return a.tiles == 2 ? launch_umma8_t<T, 128, 2>(a, tmq, st) : launch_umma8_t<T, 128, 1>(a, tmq, st);
}

}  // namespace pa
