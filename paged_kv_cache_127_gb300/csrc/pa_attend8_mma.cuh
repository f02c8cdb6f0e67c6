// pa_attend8_mma.cuh -- decode and short chunks over the 8-bit cache (the formulas
// are in pa_attend8.cuh), for calls that HBM bounds.
//
// Work.  All steps of 32 keys of all (sequence, row block, group of HG KV heads) stand in one line, and each CTA takes an
// equal stretch of it: no work list, no claims, and every CTA reads the same number of bytes.  A CTA that begins or
// ends within a (sequence, row block, group) leaves a partial (m, l, O) in the workspace; the one that takes its first
// step notes how many there are, and a second launch joins them.
//
// A CTA is a producer warp and one consumer warp per KV head of the group and 16 rows of the row block (TW of them; a
// decode: one, with 8 rows).  The producer fills a ring of steps by TMA, one box per block (all HG heads) for K and for
// V; every 32 steps, lane l looks up step l's blocks and scales.  (Warps that fill rings of their own spend 700 of 2700
// cycles a step on it: 88.6 us on 256 sequences.)  A consumer computes S = Q K^T and O += P V with mma.m16n8k16, 32 keys
// at a time.  In a decode the G <= 8 heads are rows 0-7 of A, and rows 8-15 carry the low parts of P, so that weights
// keep 22 bits; in a chunk all 16 rows are query rows.
//
// Codes come out of shared memory in 16-byte pieces with the products' dimensions and keys permuted to fit: lane
// (g, c) of a warp takes bytes 16 c .. of key row perm(g) for S (its 16 bytes are 4 k-steps), and for P V bytes
// 16 g .. of the key rows perm(2c), perm(2c + 1), whose bytes it pairs up (prmt) and converts.  perm makes both
// free of bank conflicts under the TMA swizzle (128 bytes at D 128, 64 at D 64).
#pragma once

#include <cmath>
#include <type_traits>

#include "pa_attend8.cuh"

namespace pa {

// TW: row tiles of 16 of a row block; 0: a decode (8 rows).  HG: KV heads of a CTA.
template <int D, int TW, int HG>
struct Attend8Cfg {
    static constexpr int kRows = TW ? 16 * TW : 8;           // of a row block
    static constexpr int kConsumers = HG * (TW ? TW : 1);
    static constexpr int kThreads = 32 * (kConsumers + 1);
    static constexpr int kCtas = attend8_ctas(TW, HG);       // per SM
    static constexpr int kTileBytes = kStep8 * D * HG;       // K (or V) of a step
    static constexpr int kStagesRaw = 192 * 1024 / kCtas / (2 * kTileBytes);
    static constexpr int kStages = kStagesRaw > 8 ? 8 : kStagesRaw;
    static constexpr int kNotes = HG * 32;                   // per stage (ks, log2 vs, 1 / vs, -) of two blocks and each head
    static constexpr size_t kNoteOff = (size_t)kStages * 2 * kTileBytes;
    static constexpr size_t kBarOff = kNoteOff + (size_t)kStages * kNotes;   // full and empty [kStages]
    static constexpr size_t kSmem = kBarOff + (size_t)kStages * 16 + 1024;   // + alignment slack
    static_assert(kStages >= 3, "ring");
    static_assert((kSmem + 2048) * kCtas <= 228 * 1024, "shared memory budget");
};

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

// Steps of a CTA's stretch: an equal share, but at least four (128 keys), which cost about what the launch does.
__device__ __forceinline__ long long share_of(const Attend8Args &a, long long total) {
    return max(4ll, (total + a.units - 1) / a.units);
}

// Where a warp stands in the line of steps: the sequence, row block, head group and step.
struct Place8 {
    int s, rb, h, v;
    Seq8 q;
    Steps8 st;
};

template <typename T, int D, int TW, int HG>
__global__ void __launch_bounds__(Attend8Cfg<D, TW, HG>::kThreads, Attend8Cfg<D, TW, HG>::kCtas)
    attend8_mma_kernel(const Attend8Args a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = Attend8Cfg<D, TW, HG>;
    using H = Mma16<__half>;
    constexpr int kNT = D / 8, kKS = D / 16, kRows = C::kRows, kHi = TW ? 2 : 1;  // kHi: halves of A's rows that are query rows
    constexpr int kWarps = C::kConsumers + 1;
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
            own += (long long)blocks_of(p.q) * groups * p.st.count;
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
                const long long mine = (long long)blocks_of(p.q) * groups * p.st.count;
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
    int left = (int)min(each, total - each * unit);   // steps still to take

    Place8 p;
    place_seq(p, begin_at.x, false);
    {
        const long long u = (long long)(uint32_t)begin_at.z | (long long)begin_at.w << 32;
        const long long head = u / p.st.count;
        p.v = (int)(u % p.st.count);
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
        while ((p.q.n == 0 || p.st.count == 0) && p.s + 1 < a.S);
    };
    auto first_key = [&](const Place8 &x) { return (x.v < x.st.ns ? x.v : x.v + x.st.gap) * kStep8; };

    if (warp == C::kConsumers) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = policy_evict_first();
        // per lane, of the batch's step `lane`: its blocks (-1: none) and the notes of their heads
        int z[2] = {-1, -1}, issued = 0;
        float ks[2][HG], vs[2][HG];
        bool ok = true;
        while (ok && left > 0) {
            const int n = min(left, p.st.count - p.v);
            for (int i = 0; ok && i < n; ++i, ++issued, ++p.v) {
                const int turn = i & 31;
                if (turn == 0) {
                    Place8 x = p;
                    x.v += lane;
                    const int key = first_key(x);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int k = key + b * a.B;
                        z[b] = -1;
                        if (b < nb && i + lane < n && k < p.q.len) {
                            const int pb = a.block_tables[(size_t)p.s * a.max_blocks + (k >> lb)];
                            if (pb >= 0 && pb < a.N) z[b] = pb * a.Hkv + p.h * HG;
                            else set_error(a.err, PA_DEVERR_BAD_BLOCK);
                        }
#pragma unroll
                        for (int h = 0; h < HG; ++h) {
                            ks[b][h] = z[b] >= 0 ? a.k_scales[z[b] + h] : 0.f;
                            vs[b][h] = z[b] >= 0 ? a.v_scales[z[b] + h] : -1.f;
                        }
                    }
                }
                const int st = issued % C::kStages;
                if (issued >= C::kStages) ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty(st), (uint32_t)((issued / C::kStages) - 1) & 1u, kWaitLimit));
                if (ok && lane == turn) {
                    const uint32_t at = notes + (uint32_t)(C::kNotes * st), dst = ring + (uint32_t)(st * 2 * C::kTileBytes);
#pragma unroll
                    for (int h = 0; h < HG; ++h)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int from = b < nb ? b : 0;
                            const float k1 = from ? ks[1][h] : ks[0][h], v1 = from ? vs[1][h] : vs[0][h];
                            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %3};" ::"r"(at + 32 * h + 16 * b), "f"(k1),
                                         "f"(v1 > 0.f ? lg2(v1) : 0.f), "f"(1.f / v1)
                                         : "memory");
                        }
                    const int there = (z[0] >= 0) + (z[1] >= 0);
                    if (there) mbar_arrive_expect_tx(full(st), (uint32_t)(there * 2 * a.B * D * HG));
                    else mbar_arrive(full(st));
                    if (z[0] >= 0) {
                        tma_load_3d(dst, &tmk, 0, 0, z[0], full(st), pol);
                        tma_load_3d(dst + C::kTileBytes, &tmv, 0, 0, z[0], full(st), pol);
                    }
                    if (z[1] >= 0) {
                        tma_load_3d(dst + (uint32_t)(a.B * D * HG), &tmk, 0, 0, z[1], full(st), pol);
                        tma_load_3d(dst + (uint32_t)(C::kTileBytes + a.B * D * HG), &tmv, 0, 0, z[1], full(st), pol);
                    }
                }
                __syncwarp();
            }
            left -= n;
            if (ok && left > 0) next_head(p);
        }
        if (!ok && lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
        // the shared memory outlives its copies
        for (int k = max(0, issued - C::kStages); k < issued; ++k)
            mbar_wait_bounded(full(k % C::kStages), (uint32_t)(k / C::kStages) & 1u, kWaitLimit);
        return;
    }

    // ------------------------------------------------------------ consumers
    const int head = warp % HG, member = warp / HG;        // of the group, of the row block's tiles
    const uint32_t head_at = (uint32_t)(head * a.B * D);   // of a box
    const uint32_t half_at = (uint32_t)(a.B == 16 ? 16 * D * HG : 16 * D);   // from key 0 to key 16 of a head
    bool timed_out = false;
    // the line's stretch, a (sequence, row block, group) at a time
    const int g = lane >> 2, c = lane & 3;
    int taken = 0;
    bool first_piece = true;
    while (left > 0) {
        const int n = min(left, p.st.count - p.v);           // steps of this head
        const bool whole = n == p.st.count;
        const int kvh = p.h * HG + head;
        const int r0 = p.rb * kRows + 16 * member;           // first row of the warp: row r is token r / G, head r % G
        const bool any = r0 < p.q.n * G;
        // queries as A fragments
        uint32_t qa[kKS][2 * kHi];
        float qs[kHi];                                       // scale log2(e) over the row's factor
        int pos[kHi];
#pragma unroll
        for (int hi = 0; hi < kHi; ++hi) {
            const int r = r0 + 8 * hi + g;
            const bool on = r < p.q.n * G;
            const int t = on ? r >> lg : 0;
            pos[hi] = on ? p.q.len - p.q.n + t : p.q.len - 1;
            const uint16_t *row = static_cast<const uint16_t *>(a.q) +
                                  ((size_t)(p.q.q0 + t) * a.Hq + kvh * G + (on ? r & (G - 1) : 0)) * D;
            uint32_t w[kKS][2];
#pragma unroll
            for (int ch = 0; ch < D / 64; ++ch) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (on) {
                    x = *reinterpret_cast<const uint4 *>(row + 16 * (c + 4 * ch));
                    y = *reinterpret_cast<const uint4 *>(row + 16 * (c + 4 * ch) + 8);
                }
                w[4 * ch][0] = x.x, w[4 * ch][1] = x.y, w[4 * ch + 1][0] = x.z, w[4 * ch + 1][1] = x.w;
                w[4 * ch + 2][0] = y.x, w[4 * ch + 2][1] = y.y, w[4 * ch + 3][0] = y.z, w[4 * ch + 3][1] = y.w;
            }
            float back = 1.f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = Mma16<T>::unpack(w[ks][i]);
                        top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(100, max(-100, 10 - ((int)(__float_as_uint(top) >> 23) - 127)));
                const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = Mma16<T>::unpack(w[ks][i]);
                        w[ks][i] = H::pack(v.x * up, v.y * up);
                    }
            }
            qs[hi] = a.scale * kLog2e8 * back;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                qa[ks][hi] = w[ks][0];
                qa[ks][kHi + hi] = w[ks][1];
            }
        }
        // keys that every row of the warp sees: up to its first row's position, and above its last row's window
        const int t_first = min(p.q.n - 1, r0 >> lg), t_last = min(p.q.n - 1, (r0 + (TW ? 15 : 7)) >> lg);
        const int pos_first = p.q.len - p.q.n + t_first, pos_last = p.q.len - p.q.n + t_last;
        const int seen_from = a.window > 0 ? pos_first - a.window + 1 : 0;   // below: only sinks are seen by some row
        const int whole_from = a.window > 0 ? pos_last - a.window + 1 : 0;

        float o[kNT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
        float m[kHi], l[kHi];   // m: the weights' reference (log2); l: this lane's keys only
#pragma unroll
        for (int hi = 0; hi < kHi; ++hi) m[hi] = -INFINITY, l[hi] = 0.f;

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
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(ks[b]), "=f"(lv[b]), "=f"(iv[b]), "=f"(pad) : "r"(notes + (uint32_t)(C::kNotes * st + 32 * head + 16 * b)));
                }
                const bool clear = kb + kStep8 - 1 <= pos_first && (kb >= whole_from || kb + kStep8 <= a.sinks) && iv[0] > 0.f && iv[1] > 0.f;
                // ---- S = Q K^T: 32 keys, four n-tiles of 8
                float s[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
                for (int ch = 0; ch < D / 64; ++ch) {
                    uint4 w[4];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) w[nt] = lds128(kst + (nt & 2 ? half_at : 0u) + piece8<D>(8 * (nt & 1) + perm8<D>(g), c + 4 * ch));
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) {
                        const uint32_t *q = qa[4 * ch + i4];
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt) {
                            const uint32_t x = i4 == 0 ? w[nt].x : i4 == 1 ? w[nt].y : i4 == 2 ? w[nt].z : w[nt].w;
                            H::mma(s[nt], q[0], TW ? q[kHi - 1] : 0u, q[kHi], TW ? q[2 * kHi - 1] : 0u, f16_of_codes(x & 0xffffu), f16_of_codes(x >> 16));
                        }
                    }
                }
                // this lane's bytes of its four keys' rows of V, of the first or second 16 keys
                auto load_v = [&](uint32_t (&vw)[4][D / 32], int kk) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 8 * (e >> 1) + perm8<D>(2 * c + (e & 1));
                        const uint32_t tile = vst + (kk ? half_at : 0u);
                        if constexpr (D == 128) {
                            const uint4 x = lds128(tile + piece8<D>(row, g));
                            vw[e][0] = x.x, vw[e][1] = x.y, vw[e][2] = x.z, vw[e][3] = x.w;
                        } else {
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(vw[e][0]), "=r"(vw[e][1])
                                         : "r"(tile + piece8<D>(row, g >> 1) + 8 * (g & 1)));
                        }
                        if (!clear) {  // a key that no row sees may hold anything
                            const int j = kb + 16 * kk + row;
                            if (!(iv[kk] > 0.f && j <= pos_last && (j >= seen_from || j < a.sinks))) {
#pragma unroll
                                for (int x = 0; x < D / 32; ++x) vw[e][x] = 0u;
                            }
                        }
                    }
                };
                uint32_t va[4][D / 32], vb[4][D / 32];
                load_v(va, 0);
                // ---- a_j = z_j + log2 vs, the running reference, weights
                float mx[kHi];
                bool need = false;
#pragma unroll
                for (int hi = 0; hi < kHi; ++hi) {
                    float mul[2] = {qs[hi] * ks[0], qs[hi] * ks[1]};
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) s[nt][2 * hi + e] = fmaf(s[nt][2 * hi + e], mul[nt >> 1], lv[nt >> 1]);
                }
                if (!clear) {
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = kb + 8 * nt + perm8<D>(2 * c + e);
#pragma unroll
                            for (int hi = 0; hi < kHi; ++hi)
                                if (!(iv[nt >> 1] > 0.f && j <= pos[hi] && (a.window == 0 || j > pos[hi] - a.window || j < a.sinks)))
                                    s[nt][2 * hi + e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int hi = 0; hi < kHi; ++hi) {
                    mx[hi] = fmaxf(fmaxf(fmaxf(s[0][2 * hi], s[0][2 * hi + 1]), fmaxf(s[1][2 * hi], s[1][2 * hi + 1])),
                                   fmaxf(fmaxf(s[2][2 * hi], s[2][2 * hi + 1]), fmaxf(s[3][2 * hi], s[3][2 * hi + 1])));
                    need = need || mx[hi] > m[hi] + (8.f + kLift8);
                }
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int hi = 0; hi < kHi; ++hi) {
                        float x = mx[hi];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        x = fmaxf(m[hi], x - kLift8);
                        const float alpha = x == -INFINITY ? 1.f : ex2(m[hi] - x);
                        m[hi] = x;
                        l[hi] *= alpha;
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            o[nt][2 * hi] *= alpha;
                            o[nt][2 * hi + 1] *= alpha;
                            if (TW == 0) {
                                o[nt][2] *= alpha;
                                o[nt][3] *= alpha;
                            }
                        }
                    }
                }
                uint32_t pa[2][4];   // P as A fragments of 16 keys each
#pragma unroll
                for (int hi = 0; hi < kHi; ++hi) {
                    const float mr = m[hi] == -INFINITY ? 0.f : m[hi];
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = ex2(s[2 * kk + (e >> 1)][2 * hi + (e & 1)] - mr);
                        // a block that is not there has weights of 0 (and an iv of -1)
                        l[hi] = fmaf((w[0] + w[1]) + (w[2] + w[3]), iv[kk], l[hi]);
                        pa[kk][hi] = H::pack(w[0], w[1]);
                        pa[kk][2 + hi] = H::pack(w[2], w[3]);
                        if (TW == 0) {
                            const float2 x = H::unpack(pa[kk][0]), y = H::unpack(pa[kk][2]);
                            pa[kk][1] = H::pack(w[0] - x.x, w[1] - x.y);
                            pa[kk][3] = H::pack(w[2] - y.x, w[3] - y.y);
                        }
                    }
                }
                // ---- O += P V
                load_v(vb, 1);
                auto product = [&](const uint32_t (&vw)[4][D / 32], const uint32_t (&w)[4]) {
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        const uint32_t p0 = __byte_perm(vw[0][x], vw[1][x], 0x5140), p1 = __byte_perm(vw[0][x], vw[1][x], 0x7362);
                        const uint32_t y0 = __byte_perm(vw[2][x], vw[3][x], 0x5140), y1 = __byte_perm(vw[2][x], vw[3][x], 0x7362);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t lo = e < 2 ? p0 : p1, hi = e < 2 ? y0 : y1;
                            H::mma(o[4 * x + e], w[0], w[1], w[2], w[3], f16_of_codes(e & 1 ? lo >> 16 : lo & 0xffffu),
                                   f16_of_codes(e & 1 ? hi >> 16 : hi & 0xffffu));
                        }
                    }
                };
                product(va, pa[0]);
                product(vb, pa[1]);
            }
            __syncwarp();  // every lane has read the stage
            if (lane == 0) mbar_arrive(empty(st));
            ++taken;
            ++p.v;
        }
        left -= n;
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
        for (int hi = 0; hi < kHi; ++hi) {
            float sum = l[hi];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int row = 16 * member + 8 * hi + g, r = p.rb * kRows + row;
            if (r >= p.q.n * G) continue;
            const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
            // this lane's columns: kNT from 2 kNT c on, and the kNT behind them
            float v[2][kNT];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) v[e][nt] = (TW ? o[nt][2 * hi + e] : o[nt][e] + o[nt][2 + e]) * inv;
            if (!whole) {
                float4 *to = reinterpret_cast<float4 *>(part + (size_t)row * D + 2 * kNT * c);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int x = 0; x < kNT / 4; ++x)
                        to[e * kNT / 4 + x] = make_float4(v[e][4 * x], v[e][4 * x + 1], v[e][4 * x + 2], v[e][4 * x + 3]);
                if (c == 0) *reinterpret_cast<float2 *>(part + (size_t)kRows * D + 2 * row) = make_float2(m[hi], sum);
                continue;
            }
            const size_t at = ((size_t)(p.q.q0 + (r >> lg)) * a.Hq + kvh * G + (r & (G - 1))) * D + 2 * kNT * c;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (a.out16) {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at + e * kNT);
#pragma unroll
                    for (int x = 0; x < kNT / 8; ++x)
                        to[x] = make_uint4(Mma16<T>::pack(v[e][8 * x], v[e][8 * x + 1]), Mma16<T>::pack(v[e][8 * x + 2], v[e][8 * x + 3]),
                                           Mma16<T>::pack(v[e][8 * x + 4], v[e][8 * x + 5]), Mma16<T>::pack(v[e][8 * x + 6], v[e][8 * x + 7]));
                } else {
                    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at + e * kNT);
#pragma unroll
                    for (int x = 0; x < kNT / 4; ++x) to[x] = make_float4(v[e][4 * x], v[e][4 * x + 1], v[e][4 * x + 2], v[e][4 * x + 3]);
                }
            }
        }
        first_piece = false;
        if (left > 0) next_head(p);
    }
}

// One CTA per (sequence, row block, KV head) joins its parts,
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,   M = max m_i,
// and writes the zeros of a sequence without keys.  A warp takes a row, a lane D / 32 of its columns.
template <typename T, int D, int TW, int HG>
__global__ void __launch_bounds__(128) attend8_merge_kernel(const Attend8Args a) {
    using C = Attend8Cfg<D, TW, HG>;
    constexpr int kRows = C::kRows, kPer = D / 32;
    griddep_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int G = a.Hq / a.Hkv, nrb = (a.max_query_len * G + kRows - 1) / kRows;
    const int s = blockIdx.x / (a.Hkv * nrb), h = blockIdx.x / nrb % a.Hkv, rb = blockIdx.x % nrb;
    if (!a.hdr[0]) return;
    const Seq8 q = seq_of(a, s, false);
    if (rb * kRows >= q.n * G) return;
    const bool none = q.len == 0;
    int2 note = make_int2(0, 0);
    if (!none) {
        note = reinterpret_cast<const int2 *>(a.list)[((size_t)s * (a.Hkv / HG) + h / HG) * nrb + rb];
        if (note.y == 0) return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the parts: the first in slot note.x, the others in the following CTAs' first slots
    auto part = [&](int i) { return a.parts + ((size_t)(i == 0 ? note.x : 2 * (note.x / 2 + i)) * HG + h % HG) * kRows * (D + 2); };
    for (int row = warp; row < kRows; row += 4) {
        const int r = rb * kRows + row, t = r / G;
        if (t >= q.n) break;
        float M = -INFINITY, l = 0.f, o[kPer] = {};
        for (int i = lane; i < note.y; i += 32) M = fmaxf(M, part(i)[(size_t)kRows * D + 2 * row]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        if (M == -INFINITY) M = 0.f;
#pragma unroll 4
        for (int i = 0; i < note.y; ++i) {
            const float *at = part(i);
            const float2 ml = *reinterpret_cast<const float2 *>(at + (size_t)kRows * D + 2 * row);
            const float w = ex2(ml.x - M);
            l = fmaf(w, ml.y, l);
#pragma unroll
            for (int x = 0; x < kPer; ++x) o[x] = fmaf(w, at[(size_t)row * D + kPer * lane + x], o[x]);
        }
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
    }
}

template <typename T, int D, int TW, int HG>
cudaError_t launch_attend8_t(const Attend8Args &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    using C = Attend8Cfg<D, TW, HG>;
    static std::atomic<int> configured[kMaxLaunchDevices];
    int one = 0;
    cudaError_t e = per_device_value(configured, &one, [](int, int *v) {
        *v = 1;
        return cudaFuncSetAttribute(attend8_mma_kernel<T, D, TW, HG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
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
    e = cudaLaunchKernelEx(&cfg, attend8_mma_kernel<T, D, TW, HG>, a, tmk, tmv);
    if (e != cudaSuccess) return e;
    // the join: a CTA per (sequence, KV head, row block)
    const long long blocks = ((long long)a.max_query_len * (a.Hq / a.Hkv) + C::kRows - 1) / C::kRows;
    if (blocks * a.S * a.Hkv > 0x7fffffffLL) return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)(blocks * a.S * a.Hkv));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attend8_merge_kernel<T, D, TW, HG>, a);
}

template <typename T, int D, int TW>
cudaError_t dispatch_heads(const Attend8Args &a, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    if constexpr (TW < 4)
        if (hg == 4) return launch_attend8_t<T, D, TW, 4>(a, tmk, tmv, st);
    return hg == 2 ? launch_attend8_t<T, D, TW, 2>(a, tmk, tmv, st) : launch_attend8_t<T, D, TW, 1>(a, tmk, tmv, st);
}
template <typename T, int D>
cudaError_t dispatch_attend8(const Attend8Args &a, int tw, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    switch (tw) {
        case 0: return dispatch_heads<T, D, 0>(a, hg, tmk, tmv, st);
        case 1: return dispatch_heads<T, D, 1>(a, hg, tmk, tmv, st);
        case 2: return dispatch_heads<T, D, 2>(a, hg, tmk, tmv, st);
        default: return dispatch_heads<T, D, 4>(a, hg, tmk, tmv, st);
    }
}

}  // namespace pa
