// pa_attend8_mma.cuh -- decode and short chunks over the 8-bit cache (the formulas
// are in pa_attend8.cuh), for calls that HBM bounds.
//
// Work.  All steps of 32 keys of all (sequence, row block, KV head) stand in one line, and each warp takes an equal
// stretch of it: no work list, no claims, and every warp reads the same number of bytes.  A warp that begins or
// ends within a (sequence, row block, head) leaves a partial (m, l, O) in the workspace; the warp that takes its first
// step notes how many there are, and a second launch joins them.
//
// A warp works alone: it keeps a ring of three steps in shared memory, fills it by TMA itself (lane 0, and lane 1
// for the step's second block when block_size is 16: one box per block, K and V; the block ids are read a step
// ahead, the scales come by cp.async on the same barrier), and computes S = Q K^T and O += P V with
// mma.m16n8k16.  In a decode the G <= 8 heads are rows 0-7 of A, and rows 8-15 carry the low parts of P, so
// that weights keep 22 bits; in a chunk all 16 rows are query rows.
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

constexpr int kWarps8 = 4;   // warps of a CTA

// RT: 16-row tiles of a chunk's row block; 0: a decode (8 rows).
template <int D, int RT>
struct Attend8Cfg {
    static constexpr int kRows = RT ? 16 * RT : 8;
    static constexpr int kTiles = RT ? RT : 1;
    static constexpr int kTileBytes = kStep8 * D;            // K (or V) of a step
    static constexpr int kStages = 3;
    static constexpr int kRing = kStages * 2 * kTileBytes;   // of a warp
    static constexpr int kScales = kStages * 16;             // per stage (ks, vs) of two blocks
    static constexpr size_t kScaleOff = (size_t)kWarps8 * kRing;
    static constexpr size_t kBarOff = kScaleOff + (size_t)kWarps8 * kScales;
    static constexpr size_t kSmem = kBarOff + (size_t)kWarps8 * kStages * 8 + 1024;  // + alignment slack
    static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
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

// Steps of a warp's stretch: an equal share, but at least four (128 keys), which cost about what the launch does.
__device__ __forceinline__ long long share_of(const Attend8Args &a, long long total) {
    return max(4ll, (total + a.units - 1) / a.units);
}

// Where a warp stands in the line of steps.
struct Place8 {
    int s, rb, h, v;      // sequence, row block, KV head, step
    Seq8 q;
    Steps8 st;
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kWarps8 * 32, 2)
    attend8_mma_kernel(const Attend8Args a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using C = Attend8Cfg<D, RT>;
    using H = Mma16<__half>;
    constexpr int kNT = D / 8, kKS = D / 16, kTiles = C::kTiles, kRows = C::kRows;
    extern __shared__ unsigned char smem_raw[];
    __shared__ long long sums[kWarps8];
    __shared__ int4 begin_at[kWarps8];  // (sequence, -, rest low, rest high) of each warp's first step
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.Hkv;
    const uint32_t ring = base + (uint32_t)(warp * C::kRing);
    const uint32_t scales = base + (uint32_t)(C::kScaleOff + warp * C::kScales);
    const uint32_t bars = base + (uint32_t)(C::kBarOff + warp * C::kStages * 8);
    const int nb = kStep8 / a.B, lb = __ffs(a.B) - 1;
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(bars + 8 * i, 2 * nb);
        fence_mbar_init();
        if (warp == 0) {
            prefetch_tmap(&tmk);
            prefetch_tmap(&tmv);
        }
    }
    griddep_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the line: steps of a sequence, over its row blocks and heads
    auto place_seq = [&](Place8 &p, int s, bool flag) {
        p.s = s;
        p.q = seq_of(a, s, flag);
        p.st = steps_of(a, p.q.len - p.q.n, p.q.n > 0 ? p.q.len : 0, kStep8);
    };
    auto blocks_of = [&](const Seq8 &q) { return (q.n * G + kRows - 1) / kRows; };
    long long total = 0;
    {
        const int per = (a.S + kWarps8 * 32 - 1) / (kWarps8 * 32);
        const int s0 = min(a.S, (int)threadIdx.x * per), s1 = min(a.S, s0 + per);
        long long own = 0;
        bool ok = true;
        Place8 p;
        for (int s = s0; s < s1; ++s) {
            place_seq(p, s, blockIdx.x == 0);
            ok = ok && order_ok(a, s);
            own += (long long)blocks_of(p.q) * a.Hkv * p.st.count;
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
        for (int w = 0; w < kWarps8; ++w) {
            total += sums[w];
            if (w < warp) before += sums[w];
        }
        // the thread whose sequences hold a warp's first step looks it up
        const long long each = share_of(a, total);
        for (int w = 0; w < kWarps8; ++w) {
            long long u = each * (blockIdx.x * kWarps8 + w);
            if (u < before || u >= before + own) continue;
            u -= before;
            for (int s = s0; s < s1; ++s) {
                place_seq(p, s, false);
                const long long mine = (long long)blocks_of(p.q) * a.Hkv * p.st.count;
                if (u < mine) {
                    begin_at[w] = make_int4(s, 0, (int)(u & 0xffffffffll), (int)(u >> 32));
                    break;
                }
                u -= mine;
            }
        }
        __syncthreads();
    }
    const long long each = share_of(a, total);
    const int unit = blockIdx.x * kWarps8 + warp;
    const long long u0 = each * unit;
    if (u0 >= total) return;
    int left = (int)min(each, total - u0);   // steps this warp still has to take
    const int steps = left;

    Place8 p;
    place_seq(p, begin_at[warp].x, false);
    {
        const long long u = (long long)(uint32_t)begin_at[warp].z | (long long)begin_at[warp].w << 32;
        const long long head = u / p.st.count;
        p.v = (int)(u % p.st.count);
        p.h = (int)(head % a.Hkv);
        p.rb = (int)(head / a.Hkv);
    }
    auto next_head = [&](Place8 &p) {  // the first step of the next head (there is one)
        p.v = 0;
        if (++p.h < a.Hkv) return;
        p.h = 0;
        if (++p.rb < blocks_of(p.q)) return;
        p.rb = 0;
        do place_seq(p, p.s + 1, false);
        while ((p.q.n == 0 || p.st.count == 0) && p.s + 1 < a.S);
    };

    // ---- filling the ring: lane i < nb loads block i of a step
    Place8 f = p;          // the next step to load
    int issued = 0, pb = -1;
    const uint64_t pol = policy_evict_first();
    auto first_key = [&](const Place8 &x) { return (x.v < x.st.ns ? x.v : x.v + x.st.gap) * kStep8; };
    auto look = [&]() {    // the block id of the next step to load
        if (lane < nb && issued < steps) {
            const int key = first_key(f) + lane * a.B;
            pb = key < f.q.len ? a.block_tables[(size_t)f.s * a.max_blocks + (key >> lb)] : -2;
        }
    };
    look();
    auto fill = [&]() {
        if (issued >= steps) return;
        const int st = issued % C::kStages;
        if (lane < nb) {
            const uint32_t bar = bars + 8 * st;
            const uint32_t sc = scales + 16 * st + 8 * lane;
            if (pb >= 0 && pb < a.N) {
                const uint32_t dst = ring + (uint32_t)(st * 2 * C::kTileBytes + lane * a.B * D);
                const int z = pb * a.Hkv + f.h;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sc), "l"(a.k_scales + z) : "memory");
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sc + 4), "l"(a.v_scales + z) : "memory");
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
                mbar_arrive_expect_tx(bar, (uint32_t)(2 * a.B * D));
                tma_load_3d(dst, &tmk, 0, 0, z, bar, pol);
                tma_load_3d(dst + C::kTileBytes, &tmv, 0, 0, z, bar, pol);
            } else {
                if (pb != -2) set_error(a.err, PA_DEVERR_BAD_BLOCK);
                // no block: its keys are masked by a scale that no block has
                asm volatile("st.shared.v2.f32 [%0], {%1, %1};" ::"r"(sc), "f"(-1.f) : "memory");
                mbar_arrive(bar);
                mbar_arrive(bar);
            }
        }
        ++issued;
        if (++f.v == f.st.count && issued < steps) next_head(f);
        look();
    };
    __syncwarp();
    for (int i = 0; i < C::kStages; ++i) fill();

    // ---- the line's stretch, a (sequence, row block, head) at a time
    const int g = lane >> 2, c = lane & 3;
    int taken = 0;
    bool first_piece = true;
    while (left > 0) {
        const int n = min(left, p.st.count - p.v);           // steps of this head
        const bool whole = n == p.st.count;
        const int r0 = p.rb * kRows;                         // first row of the block: row r is token r / G, head r % G
        // queries as A fragments
        uint32_t qa[kTiles][kKS][4];
        float qs[kTiles][2];                                 // scale log2(e) over the row's factor
        int pos[kTiles][2];
#pragma unroll
        for (int rt = 0; rt < kTiles; ++rt) {
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                if (RT == 0 && hi) {
#pragma unroll
                    for (int ks = 0; ks < kKS; ++ks) qa[rt][ks][1] = qa[rt][ks][3] = 0u;
                    qs[rt][1] = 0.f;
                    pos[rt][1] = pos[rt][0];
                    continue;
                }
                const int r = r0 + 16 * rt + 8 * hi + g;
                const bool on = r < p.q.n * G;
                const int t = on ? r / G : 0;
                pos[rt][hi] = on ? p.q.len - p.q.n + t : p.q.len - 1;
                const uint16_t *row = static_cast<const uint16_t *>(a.q) +
                                      ((size_t)(p.q.q0 + t) * a.Hq + p.h * G + (on ? r - t * G : 0)) * D;
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
                qs[rt][hi] = a.scale * kLog2e8 * back;
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks) {
                    qa[rt][ks][hi] = w[ks][0];
                    qa[rt][ks][2 + hi] = w[ks][1];
                }
            }
        }
        // keys that every row of the block sees: up to its first row's position, and above its last row's window
        const int t_first = r0 / G, t_last = min(p.q.n - 1, (r0 + kRows - 1) / G);
        const int pos_first = p.q.len - p.q.n + t_first, pos_last = p.q.len - p.q.n + t_last;
        const int seen_from = a.window > 0 ? pos_first - a.window + 1 : 0;   // below: only sinks are seen by some row
        const int whole_from = a.window > 0 ? pos_last - a.window + 1 : 0;

        float o[kTiles][kNT][4];
#pragma unroll
        for (int rt = 0; rt < kTiles; ++rt)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) o[rt][nt][0] = o[rt][nt][1] = o[rt][nt][2] = o[rt][nt][3] = 0.f;
        float m[kTiles][2], l[kTiles][2];   // m: the weights' reference (log2); l: this lane's keys only
#pragma unroll
        for (int rt = 0; rt < kTiles; ++rt) m[rt][0] = m[rt][1] = -INFINITY, l[rt][0] = l[rt][1] = 0.f;
        bool timed_out = false;

        for (int i = 0; i < n; ++i) {
            const int st = taken % C::kStages;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bars + 8 * st, (uint32_t)(taken / C::kStages) & 1u, kWaitLimit))) {
                timed_out = true;
                break;
            }
            const int kb = first_key(p);
            const uint32_t kst = ring + (uint32_t)(st * 2 * C::kTileBytes), vst = kst + C::kTileBytes;
            float2 sc[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(sc[b].x), "=f"(sc[b].y) : "r"(scales + 16 * st + (b < nb ? 8 * b : 0)));
            const bool clear = kb + kStep8 - 1 <= pos_first && (kb >= whole_from || kb + kStep8 <= a.sinks) && sc[0].y > 0.f && sc[1].y > 0.f;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const float ks = kk ? sc[1].x : sc[0].x, vs = kk ? sc[1].y : sc[0].y;
                const float lv = lg2(vs), ivs = 1.f / vs;
                // ---- S = Q K^T: 16 keys, two n-tiles of 8
                float s[kTiles][2][4];
#pragma unroll
                for (int rt = 0; rt < kTiles; ++rt)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) s[rt][nt][0] = s[rt][nt][1] = s[rt][nt][2] = s[rt][nt][3] = 0.f;
#pragma unroll
                for (int ch = 0; ch < D / 64; ++ch) {
                    uint4 w[2];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) w[nt] = lds128(kst + piece8<D>(16 * kk + 8 * nt + perm8<D>(g), c + 4 * ch));
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const uint32_t x = i4 == 0 ? w[nt].x : i4 == 1 ? w[nt].y : i4 == 2 ? w[nt].z : w[nt].w;
                            const uint32_t b0 = f16_of_codes(x & 0xffffu), b1 = f16_of_codes(x >> 16);
#pragma unroll
                            for (int rt = 0; rt < kTiles; ++rt) {
                                const uint32_t *q = qa[rt][4 * ch + i4];
                                H::mma(s[rt][nt], q[0], q[1], q[2], q[3], b0, b1);
                            }
                        }
                }
                // ---- a_j = z_j + log2 vs, masks, the running reference, weights
                uint32_t pa[kTiles][4];
                bool need = false;
                float mx[kTiles][2];
#pragma unroll
                for (int rt = 0; rt < kTiles; ++rt)
#pragma unroll
                    for (int hi = 0; hi < (RT ? 2 : 1); ++hi) {
                        const float mul = qs[rt][hi] * ks;
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float &x = s[rt][nt][2 * hi + e];
                                x = fmaf(x, mul, lv);
                                if (!clear) {
                                    const int j = kb + 16 * kk + 8 * nt + perm8<D>(2 * c + e);
                                    const bool seen = vs > 0.f && j <= pos[rt][hi] && (a.window == 0 || j > pos[rt][hi] - a.window || j < a.sinks);
                                    if (!seen) x = -INFINITY;
                                }
                            }
                        mx[rt][hi] = fmaxf(fmaxf(s[rt][0][2 * hi], s[rt][0][2 * hi + 1]), fmaxf(s[rt][1][2 * hi], s[rt][1][2 * hi + 1]));
                        need = need || mx[rt][hi] > m[rt][hi] + (8.f + kLift8);
                    }
                if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                    for (int rt = 0; rt < kTiles; ++rt)
#pragma unroll
                        for (int hi = 0; hi < (RT ? 2 : 1); ++hi) {
                            float x = mx[rt][hi];
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            x = fmaxf(m[rt][hi], x - kLift8);
                            const float alpha = x == -INFINITY ? 1.f : ex2(m[rt][hi] - x);
                            m[rt][hi] = x;
                            l[rt][hi] *= alpha;
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt) {
                                o[rt][nt][2 * hi] *= alpha;
                                o[rt][nt][2 * hi + 1] *= alpha;
                                if (RT == 0) {
                                    o[rt][nt][2] *= alpha;
                                    o[rt][nt][3] *= alpha;
                                }
                            }
                        }
                }
#pragma unroll
                for (int rt = 0; rt < kTiles; ++rt)
#pragma unroll
                    for (int hi = 0; hi < (RT ? 2 : 1); ++hi) {
                        const float mr = m[rt][hi] == -INFINITY ? 0.f : m[rt][hi];
                        float w[4], sum = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            w[e] = ex2(s[rt][e >> 1][2 * hi + (e & 1)] - mr);
                            sum += w[e];
                        }
                        l[rt][hi] = clear || vs > 0.f ? fmaf(sum, ivs, l[rt][hi]) : l[rt][hi];
                        pa[rt][hi] = H::pack(w[0], w[1]);
                        pa[rt][2 + hi] = H::pack(w[2], w[3]);
                        if (RT == 0) {
                            const float2 x = H::unpack(pa[rt][0]), y = H::unpack(pa[rt][2]);
                            pa[rt][1] = H::pack(w[0] - x.x, w[1] - x.y);
                            pa[rt][3] = H::pack(w[2] - y.x, w[3] - y.y);
                        }
                    }
                // ---- O += P V
                uint32_t vw[4][D / 32];   // this lane's bytes of its four keys' rows
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 16 * kk + 8 * (e >> 1) + perm8<D>(2 * c + (e & 1));
                    if constexpr (D == 128) {
                        const uint4 x = lds128(vst + piece8<D>(row, g));
                        vw[e][0] = x.x, vw[e][1] = x.y, vw[e][2] = x.z, vw[e][3] = x.w;
                    } else {
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(vw[e][0]), "=r"(vw[e][1])
                                     : "r"(vst + piece8<D>(row, g >> 1) + 8 * (g & 1)));
                    }
                    if (!clear) {  // a key that no row sees may hold anything
                        const int j = kb + row;
                        if (!(vs > 0.f && j <= pos_last && (j >= seen_from || j < a.sinks))) {
#pragma unroll
                            for (int x = 0; x < D / 32; ++x) vw[e][x] = 0u;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint32_t p0 = __byte_perm(vw[0][x], vw[1][x], 0x5140), p1 = __byte_perm(vw[0][x], vw[1][x], 0x7362);
                    const uint32_t y0 = __byte_perm(vw[2][x], vw[3][x], 0x5140), y1 = __byte_perm(vw[2][x], vw[3][x], 0x7362);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = e < 2 ? p0 : p1, hi = e < 2 ? y0 : y1;
                        const uint32_t b0 = f16_of_codes(e & 1 ? lo >> 16 : lo & 0xffffu), b1 = f16_of_codes(e & 1 ? hi >> 16 : hi & 0xffffu);
#pragma unroll
                        for (int rt = 0; rt < kTiles; ++rt) H::mma(o[rt][4 * x + e], pa[rt][0], pa[rt][1], pa[rt][2], pa[rt][3], b0, b1);
                    }
                }
            }
            ++taken;
            ++p.v;
            __syncwarp();  // every lane has read the stage
            fill();
        }
        left -= n;
        if (timed_out) {
            if (lane == 0) set_error(a.err, PA_DEVERR_TIMEOUT);
            break;
        }

        // ---- the outputs, or this warp's part of them
        const bool starts = p.v == n;          // this warp took the head's first step
        const int slot = first_piece ? 2 * unit : 2 * unit + 1;
        float *part = a.parts + (size_t)slot * kRows * (D + 2);
        int2 *notes = reinterpret_cast<int2 *>(a.list) + ((size_t)p.s * a.Hkv + p.h) * ((a.max_query_len * G + kRows - 1) / kRows) + p.rb;
        if (starts && lane == 0) {
            // the head's steps from here on: this warp's n, then the following warps'
            const int rest = p.st.count - n;
            *notes = make_int2(slot, whole ? 0 : 1 + (int)((rest + each - 1) / each));
        }
#pragma unroll
        for (int rt = 0; rt < kTiles; ++rt)
#pragma unroll
            for (int hi = 0; hi < (RT ? 2 : 1); ++hi) {
                float sum = l[rt][hi];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int row = 16 * rt + 8 * hi + g, r = r0 + row;
                if (r >= p.q.n * G) continue;
                const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                // this lane's columns: kNT from 2 kNT c on, and the kNT behind them
                float v[2][kNT];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) v[e][nt] = (RT ? o[rt][nt][2 * hi + e] : o[rt][nt][e] + o[rt][nt][2 + e]) * inv;
                if (!whole) {
                    float4 *to = reinterpret_cast<float4 *>(part + (size_t)row * D + 2 * kNT * c);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int x = 0; x < kNT / 4; ++x)
                            to[e * kNT / 4 + x] = make_float4(v[e][4 * x], v[e][4 * x + 1], v[e][4 * x + 2], v[e][4 * x + 3]);
                    if (c == 0) *reinterpret_cast<float2 *>(part + (size_t)kRows * D + 2 * row) = make_float2(m[rt][hi], sum);
                    continue;
                }
                const int t = r / G;
                const size_t at = ((size_t)(p.q.q0 + t) * a.Hq + p.h * G + (r - t * G)) * D + 2 * kNT * c;
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
    // the shared memory outlives its copies
    for (int k = taken; k < issued; ++k) mbar_wait_bounded(bars + 8 * (k % C::kStages), (uint32_t)(k / C::kStages) & 1u, kWaitLimit);
}

// One CTA per (sequence, row block, KV head) joins its parts,
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,   M = max m_i,
// and writes the zeros of a sequence without keys.  A warp takes a row, a lane D / 32 of its columns.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(128) attend8_merge_kernel(const Attend8Args a) {
    using C = Attend8Cfg<D, RT>;
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
        note = reinterpret_cast<const int2 *>(a.list)[blockIdx.x];
        if (note.y == 0) return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the parts: the first in slot note.x, the others in the following warps' first slots
    auto part = [&](int i) { return a.parts + (size_t)(i == 0 ? note.x : 2 * (note.x / 2 + i)) * kRows * (D + 2); };
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

template <typename T, int D, int RT>
cudaError_t launch_attend8_t(const Attend8Args &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    using C = Attend8Cfg<D, RT>;
    static std::atomic<int> configured[kMaxLaunchDevices];
    int one = 0;
    const cudaError_t e = per_device_value(configured, &one, [](int, int *v) {
        *v = 1;
        return cudaFuncSetAttribute(attend8_mma_kernel<T, D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.units + kWarps8 - 1) / kWarps8));
    cfg.blockDim = dim3(kWarps8 * 32);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend8_mma_kernel<T, D, RT>, a, tmk, tmv);
}

template <typename T, int D, int RT>
cudaError_t launch_merge8_t(const Attend8Args &a, cudaStream_t st) {
    const int G = a.Hq / a.Hkv, rows = Attend8Cfg<D, RT>::kRows;
    const long long ctas = (long long)a.S * a.Hkv * ((a.max_query_len * (long long)G + rows - 1) / rows);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend8_merge_kernel<T, D, RT>, a);
}

// The launches of one query type.
template <typename T>
cudaError_t dispatch_attend8(const Attend8Args &a, int row_tiles, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    if (a.D == 64)
        return row_tiles == 0   ? launch_attend8_t<T, 64, 0>(a, tmk, tmv, st)
               : row_tiles == 1 ? launch_attend8_t<T, 64, 1>(a, tmk, tmv, st)
                                : launch_attend8_t<T, 64, 2>(a, tmk, tmv, st);
    return row_tiles == 0   ? launch_attend8_t<T, 128, 0>(a, tmk, tmv, st)
           : row_tiles == 1 ? launch_attend8_t<T, 128, 1>(a, tmk, tmv, st)
                            : launch_attend8_t<T, 128, 2>(a, tmk, tmv, st);
}
template <typename T>
cudaError_t dispatch_merge8(const Attend8Args &a, int row_tiles, cudaStream_t st) {
    if (a.D == 64)
        return row_tiles == 0   ? launch_merge8_t<T, 64, 0>(a, st)
               : row_tiles == 1 ? launch_merge8_t<T, 64, 1>(a, st)
                                : launch_merge8_t<T, 64, 2>(a, st);
    return row_tiles == 0   ? launch_merge8_t<T, 128, 0>(a, st)
           : row_tiles == 1 ? launch_merge8_t<T, 128, 1>(a, st)
                            : launch_merge8_t<T, 128, 2>(a, st);
}

}  // namespace pa
