// pa_write8.cu -- rotary positions of new queries and keys, and the write of keys
// and values into a cache of e4m3 codes with one scale per (block, KV head).
//
// A value x of a block is stored as code(x / s), s the block's scale for that head: the smallest power of
// two 2^e >= 2^-40 with max |x| <= 448 2^e over the block's values, for keys max |x| <= 316 2^e of the values
// before their rotation (which grows a value by sqrt(2) at most).  A floating code's relative error does not depend
// on its scale, so a power of two costs nothing in precision and makes everything around it exact: the division by s,
// the products of attention with s, and the step from one scale to a larger one when a block's later tokens are
// louder (a code only loses bits where it becomes subnormal).  The bound before the rotation makes the scale a
// function of the 16-bit inputs alone.
//
// Work.  Two kinds of CTAs in one launch.  One kind takes keys and values: the tokens of one block stand next to each
// other in the list (a run), and a CTA takes the runs that start among its tile of 16 tokens, for some of the KV heads,
// one after the other (at D 64 two at a time), so a block's scale has one writer.  Sixteen rows of a head's keys
// and values stay in registers from the maxima, through the scales, to the codes, while the next head's are on their way;
// further rows (runs may begin anywhere in a tile) are read again.  Rows that a block held before are rescaled by the
// same CTA where the scale grew.  The other kind turns the queries of two tokens each, as the write into a 16-bit cache
// does.  First loads are under way before the angles are computed (as in pa_rope.cuh, once per (row, pair), in shared memory).
// (Queries in the same CTAs as their KV head: 63 us instead of 39 for 8192 tokens of 32 + 8 heads, as each head then pays for the angles.)
//
// Bound: HBM for a prompt (each q element read and written, each k, v element read as 16 bits and written
// as 8), latency for a step.
// Measured: 8192 tokens of 32 + 8 heads (D 128, bf16) turned in whole halves 38 us (floor 27), as neighbours 37, 64 of 128
// elements 37, in halves that are not whole units (36 elements, partners read one by one) 108; 256 tokens 7.7, one 4.2;
// pa_write_kv8 17 and 4.3.  Seven CTAs an SM leave 72 registers, with 48 to 76 bytes a thread spilled in whole halves.
#include "pa_device.cuh"
#include "pa_kv8.h"
#include "pa_mma.cuh"
#include "pa_rope.cuh"

namespace pa {

namespace {

constexpr int kThreads8 = 128;
constexpr int kTile = 16;          // tokens of a CTA's tile, and rows of a pass
constexpr int kRows = kTile + 32;  // rows of the runs that start in it, at most (block_size <= 32)

enum Pairing { kHalves, kNeighbours, kSplit };  // kSplit: halves that are not whole units of 8

// Two fp32 values as e4m3 codes (x0 in the low byte); what is infinite becomes NaN.
__device__ __forceinline__ uint32_t codes2(float x0, float x1) {
    uint16_t r;
    x0 += x0 - x0;
    x1 += x1 - x1;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
    return r;
}
__device__ __forceinline__ float2 values2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return Mma16<__half>::unpack(h);
}

template <typename T>
struct Bits16;
template <>
struct Bits16<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7f80u;
    static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
};
template <>
struct Bits16<__half> {
    static constexpr uint32_t kInf = 0x7c00u;
    static __device__ __forceinline__ float value(uint32_t b) { return Mma16<__half>::unpack(b).x; }
};

// Largest finite |x| of two units, as bits.
template <typename T>
__device__ __forceinline__ uint32_t loudest(const uint4 &x, const uint4 &y) {
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    uint32_t r = max(m & 0xffffu, m >> 16);
    if (r >= Bits16<T>::kInf) {  // infinities and NaN do not count
        r = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
            if (lo < Bits16<T>::kInf) r = max(r, lo);
            if (hi < Bits16<T>::kInf) r = max(r, hi);
        }
    }
    return r;
}

// The smallest power of two >= 2^kScaleFloor whose `most`-fold (most = c 2^8, 1 < c < 2) holds x.
__device__ __forceinline__ float scale_of(float x, float most) {
    const uint32_t b = __float_as_uint(x);
    const float m = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);  // x = m 2^k
    const int k = (int)(b >> 23) - 127;
    int e = k - 8 + (m > most * 0x1p-8f ? 1 : 0);
    e = max(e, kScaleFloor);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// What a thread has of a head: two units of 8 elements, u0 and u0 + du, that turn with each other or each with itself.
template <typename T, int D, int kPairing>
struct Part8 {
    static constexpr int L = D / 16;                                                     // lanes of a row
    static constexpr int kA = kPairing == kHalves ? 8 : kPairing == kNeighbours ? 4 : 1;  // pairs of a unit
    // (cos, sin) of a row: those that one thread needs kCols apart, rows off each other by some banks
    static constexpr int kCols = D / 2 / kA, kRow = D / 2 + 8;
    static constexpr int kW = kPairing == kSplit ? 1 : 8;
    int R, half, c, u0, du;
    bool turns;   // kHalves: whether the units are a pair that turns
    __device__ __forceinline__ Part8(int R_, int lane) : R(R_), half(R_ / 2), c(lane) {
        const int turning = half / 8;
        turns = kPairing != kHalves || c < turning;
        u0 = kPairing == kHalves ? (turns ? 8 * c : R + 8 * (c - turning)) : 8 * c;
        du = kPairing == kHalves ? (turns ? half : (D - R) / 2) : D / 2;
    }
    static __device__ __forceinline__ int place(int r, int p) { return r * kRow + p % kA * kCols + p / kA; }
    __device__ __forceinline__ void load(const T *head, uint4 &x, uint4 &y) const {
        x = *reinterpret_cast<const uint4 *>(head + u0);
        y = *reinterpret_cast<const uint4 *>(head + u0 + du);
    }
    // its pairs' (cos, sin) of row r
    __device__ __forceinline__ void angles(const float2 *cs, int r, float2 (&w)[kW]) const {
        if (half == 0) return;  // nothing turns, and no angles were computed
        if constexpr (kPairing == kHalves) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = cs[r * kRow + e * kCols + (turns ? c : 0)];
        } else if constexpr (kPairing == kNeighbours) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = cs[r * kRow + (e & 3) * kCols + (e < 4 ? c : c + L)];
        }
    }
    // The 16 values, turned by w (kSplit: by row r of cs).  (x, y) are its units, `head` where they come from.
    __device__ __forceinline__ void turn(const uint4 &x, const uint4 &y, const T *head, const float2 *cs, int r,
                                         const float2 (&w)[kW], float (&f)[16]) const {
        Elem<T>::unpack(x, f);
        Elem<T>::unpack(y, f + 8);
        if constexpr (kPairing == kHalves) {
            if (turns) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 t = turned(f[e], f[8 + e], w[e]);
                    f[e] = t.x, f[8 + e] = t.y;
                }
            }
        } else if constexpr (kPairing == kNeighbours) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int p = (e < 4 ? u0 : u0 + du) / 2 + (e & 3);
                if (p < half) {
                    const float2 t = turned(f[2 * e], f[2 * e + 1], w[e]);
                    f[2 * e] = t.x, f[2 * e + 1] = t.y;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int d = (e < 8 ? u0 : u0 + du) + (e & 7);
                if (d < R) {
                    const bool low = d < half;
                    const float2 t = cs[r * kRow + (low ? d : d - half)];
                    const float other = static_cast<float>(head[low ? d + half : d - half]);
                    f[e] = low ? turned(f[e], other, t).x : turned(other, f[e], t).y;
                }
            }
        }
    }
};

// The queries of tokens t0, t0 + 1, every parts-th round of their heads.
template <typename T, int D, int kPairing>
__device__ __forceinline__ void turn_queries(const Write8Args &a, int t0, int part, int parts, float2 *cs) {
    using P = Part8<T, D, kPairing>;
    constexpr int kU = 4, kStep = kThreads8 / P::L;   // heads of a thread in flight; heads of a round
    const P my(a.R, threadIdx.x % P::L);
    const int nt = min(2, a.T - t0), all = nt * a.Hq, step = kStep * parts;
    auto head = [&](int m) { return static_cast<const T *>(a.q) + (size_t)(t0 + (m >= a.Hq)) * a.q_stride + (size_t)(m >= a.Hq ? m - a.Hq : m) * D; };
    uint4 x[kU], y[kU];
    auto load = [&](int m0) {
#pragma unroll
        for (int u = 0; u < kU; ++u) my.load(head(min(m0 + u * step, all - 1)), x[u], y[u]);  // past the end: what others load
    };
    const int m0 = part * kStep + threadIdx.x / P::L;
    load(m0);
    bool on[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t slot = t < nt ? a.slots[t0 + t] : -1;
        on[t] = slot >= 0 && slot < (int64_t)a.N * a.B;   // (the CTAs of keys and values report the others)
    }
    for (int e = threadIdx.x; e < nt * my.half; e += kThreads8) {
        const int r = e / my.half, p = e - r * my.half;
        cs[P::place(r, p)] = turn_at(turn_fraction(a.freqs[p]), pair_position(a, t0 + r, p), a.mscale);
    }
    __syncthreads();
    for (int m1 = m0; m1 - (int)threadIdx.x / P::L < all; m1 += kU * step) {   // the same rounds for the whole CTA
        if (m1 != m0) load(m1);
        float2 w[P::kW];
        int row = -1;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int m = min(m1 + u * step, all - 1), r = m >= a.Hq;
            if (r != row) my.angles(cs, row = r, w);
            float f[16];
            my.turn(x[u], y[u], head(m), cs, r, w, f);
            x[u] = make_uint4(Mma16<T>::pack(f[0], f[1]), Mma16<T>::pack(f[2], f[3]), Mma16<T>::pack(f[4], f[5]), Mma16<T>::pack(f[6], f[7]));
            y[u] = make_uint4(Mma16<T>::pack(f[8], f[9]), Mma16<T>::pack(f[10], f[11]), Mma16<T>::pack(f[12], f[13]), Mma16<T>::pack(f[14], f[15]));
        }
        __syncwarp();  // q_out may be q: the lanes of a head have read it
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int m = m1 + u * step;
            if (m >= all || !(m >= a.Hq ? on[1] : on[0])) continue;
            T *to = static_cast<T *>(a.q_out) + (size_t)(t0 + (m >= a.Hq)) * a.q_out_stride + (size_t)(m >= a.Hq ? m - a.Hq : m) * D + my.u0;
            *reinterpret_cast<uint4 *>(to) = x[u];
            *reinterpret_cast<uint4 *>(to + my.du) = y[u];
        }
    }
}

// grid: tiles * kv_parts CTAs of keys and values, which take longest, then those of the queries, q_parts for two tokens.
template <typename T, int D, int kPairing>
__global__ void __launch_bounds__(kThreads8, kPairing == kSplit ? 3 : 7) write8_kernel(const Write8Args a, int kv_parts, int q_parts) {
    using P = Part8<T, D, kPairing>;
    constexpr int L = P::L;
    constexpr int kHeads = kThreads8 / (kTile * L);  // KV heads at a time: 1 (D 128) or 2
    extern __shared__ float2 cs[];
    __shared__ unsigned long long fractions[D / 2];   // of a turn, per pair: fp64 work, once a CTA
    __shared__ int64_t slots[kRows + 2];
    __shared__ uint32_t top[2][kRows][2 * kHeads];  // per run: its loudest value of K and of V (bits), for heads in turn
    __shared__ float inv[kRows][2 * kHeads];        // per run: 1 / scale
    __shared__ float ratio[kRows][2 * kHeads];      // per run: old scale / new where the block's earlier rows change, else 1
    __shared__ int run_row[kRows], run_off[kRows];  // per run: its first row, and the first slot of its block that it takes
    __shared__ int grown[2];                        // whether some ratio is not 1, for heads in turn
    const int tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int kv_ctas = (a.T + kTile - 1) / kTile * kv_parts;
    if ((int)blockIdx.x >= kv_ctas) {
        const int i = blockIdx.x - kv_ctas;
        turn_queries<T, D, kPairing>(a, i / q_parts * 2, i % q_parts, q_parts, cs);
        return;
    }

    // ---- the runs that start in the tile: slots[j] is token t0 + j - 1
    const P my(a.R, tid % L);
    const int half = my.half;
    const int t0 = (int)(blockIdx.x / kv_parts) * kTile, span = kTile + a.B;
    if (tid < half) fractions[tid] = turn_fraction(a.freqs[tid]);
    if (tid <= span) {
        const int t = t0 + tid - 1;
        int64_t slot = t >= 0 && t < a.T ? a.slots[t] : -1;
        if (slot >= (int64_t)a.N * a.B) {
            set_error(a.err, PA_DEVERR_BAD_SLOT);
            slot = -1;
        }
        slots[tid] = slot;
    }
    __syncthreads();
    const int lb = __ffs(a.B) - 1;  // block_size is a power of two
    auto starts = [&](int j) {  // whether token t0 + j begins a run (padding and the list's end do)
        if (j >= span) return false;
        return t0 + j == 0 || slots[j + 1] < 0 || slots[j] < 0 || (slots[j + 1] >> lb) != (slots[j] >> lb);
    };
    const uint64_t mask = (uint64_t)__ballot_sync(0xffffffffu, starts(lane)) |
                          (uint64_t)__ballot_sync(0xffffffffu, starts(lane + 32)) << 32;
    const uint64_t mine = mask & ((1ull << kTile) - 1ull);
    if (mine == 0) return;
    const int first = __ffsll((long long)mine) - 1;
    const uint64_t behind = mask >> kTile;
    const int rows = min(a.T - t0, behind ? kTile + __ffsll((long long)behind) - 1 : span - 1) - first;
    if (rows <= 0) return;
    auto begins = [&](int r) { return (mask >> (first + r) & 1ull) != 0; };
    auto run_of = [&](int r) { return __popcll((mask >> first) & ((2ull << r) - 1ull)) - 1; };
    auto slot_of = [&](int r) { return slots[1 + first + r]; };
    const int tok0 = t0 + first;

    // ---- what the runs are, once for all heads
    const int runs = __popcll((mask >> first) & ((1ull << rows) - 1ull));
    if (tid < rows && begins(tid)) {
        const int run = run_of(tid);
        int off = 0;
        if (slot_of(tid) >= 0) {
            off = (int)(slot_of(tid) & (a.B - 1));
            for (int n = tid + 1; n < rows && !begins(n); ++n) off = min(off, (int)(slot_of(n) & (a.B - 1)));
        }
        run_row[run] = tid;
        run_off[run] = off;
    }
    for (int i = tid; i < runs * 2 * kHeads; i += kThreads8) top[0][i / (2 * kHeads)][i % (2 * kHeads)] = 0u;
    if (tid < 2) grown[tid] = 0;

    // ---- a thread's row of a pass, and its KV head h (of the part's, kHeads at a time)
    const int prow = tid / L % kTile, own = tid / (kTile * L), c = my.c, prun = prow < rows ? run_of(prow) : 0;
    const int per = (a.Hkv + kv_parts - 1) / kv_parts, h0 = (int)(blockIdx.x % kv_parts) * per, h_end = min(a.Hkv, h0 + per);
    auto k_row = [&](int r, int h) { return static_cast<const T *>(a.k) + (size_t)(tok0 + r) * a.k_stride + (size_t)h * D; };
    auto v_row = [&](int r, int h) { return static_cast<const T *>(a.v) + (size_t)(tok0 + r) * a.v_stride + (size_t)h * D; };
    // the first pass's rows of a head (threads past the rows or heads load what others do, so that nothing branches around a load)
    uint4 kx, ky, vx, vy, kx1, ky1, vx1, vy1;
    auto fetch = [&](int h, uint4 &k0, uint4 &k1, uint4 &v0, uint4 &v1) {
        const int r = min(prow, rows - 1);
        h = min(h, a.Hkv - 1);
        my.load(k_row(r, h), k0, k1);
        my.load(v_row(r, h), v0, v1);
    };
    if (h0 >= h_end) return;
    fetch(h0 + own, kx, ky, vx, vy);
    for (int e = tid; e < rows * half; e += kThreads8) {
        const int r = e / half, p = e - r * half;
        cs[P::place(r, p)] = turn_at(fractions[p], pair_position(a, tok0 + r, p), a.mscale);
    }
    __syncthreads();
    auto loudest_of_row = [&](const uint4 &x, const uint4 &y) {
        uint32_t m = loudest<T>(x, y);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    };

    // thread i: run i / (2 kHeads), of head own_i, K or V
    const int run_i = tid / (2 * kHeads), which_i = tid & 1, own_i = (tid >> 1) % kHeads;
    auto scale_at = [&](int run, int which, int h) {
        return (which ? a.v_scales : a.k_scales) + (size_t)(slot_of(run_row[run]) >> lb) * a.Hkv + h;
    };
    auto old_of = [&](int hb) {   // the old scale of this thread's run and head, where it counts
        if (run_i >= runs || hb + own_i >= h_end || slot_of(run_row[run_i]) < 0 || run_off[run_i] == 0) return 0.f;
        return *scale_at(run_i, which_i, hb + own_i);
    };
    float old = old_of(h0);
    int turn_of = 0;
    for (int hb = h0; hb < h_end; hb += kHeads, turn_of ^= 1) {
        const int h = hb + own;
        const bool live = h < h_end;
        // ---- the loudest value of each run
        for (int r = prow; r < (rows + kTile - 1) / kTile * kTile; r += kTile) {
            uint4 x = kx, y = ky, z = vx, w = vy;
            const bool here = r < rows && live;
            if (r >= kTile && here) {
                my.load(k_row(r, h), x, y);
                my.load(v_row(r, h), z, w);
            }
            const uint32_t mk = loudest_of_row(x, y), mv = loudest_of_row(z, w);
            if (c < 2 && here) atomicMax(&top[turn_of][r < kTile ? prun : run_of(r)][2 * own + c], c ? mv : mk);
        }
        if (hb + kHeads < h_end) fetch(h + kHeads, kx1, ky1, vx1, vy1);
        __syncthreads();

        // ---- the scales of each run, and the next head's maxima set back
        for (int i = tid; i < runs * 2 * kHeads; i += kThreads8) {
            const int run = i / (2 * kHeads), which = i & 1, o = (i >> 1) % kHeads;
            const uint32_t m = top[turn_of][run][i % (2 * kHeads)];
            top[turn_of ^ 1][run][i % (2 * kHeads)] = 0u;
            if (hb + o >= h_end || slot_of(run_row[run]) < 0) continue;
            const float x = Bits16<T>::value(m);
            float s = which || half == 0 ? scale_of(x, kLoudestPlain) : scale_of(x * fmaxf(1.f, fabsf(a.mscale)), kLoudestTurned);
            float grew = 1.f;
            float *at = scale_at(run, which, hb + o);
            if (run_off[run] > 0) {
                const float was = i == tid ? old : *at;
                if (was < s) grew = was / s;
                else s = fmaxf(was, s);  // an old scale that is no number counts as none
            }
            *at = s;
            inv[run][i % (2 * kHeads)] = 1.f / s;
            ratio[run][i % (2 * kHeads)] = grew;
            if (grew != 1.f) grown[turn_of] = 1;
        }
        if (tid == 0) grown[turn_of ^ 1] = 0;
        if (hb + kHeads < h_end) old = old_of(hb + kHeads);
        __syncthreads();

        // ---- keys and values
        for (int r = prow; r < rows && live; r += kTile) {
            const int64_t slot = slot_of(r);
            if (slot < 0) continue;
            if (r >= kTile) {
                my.load(k_row(r, h), kx, ky);
                my.load(v_row(r, h), vx, vy);
            }
            const int run = r < kTile ? prun : run_of(r);
            const size_t at = (((size_t)(slot >> lb) * a.Hkv + h) * a.B + (size_t)(slot & (a.B - 1))) * D;
            float f[16];
            auto store = [&](uint8_t *row, float s) {
                uint32_t p[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = codes2(f[2 * e] * s, f[2 * e + 1] * s);
                *reinterpret_cast<uint2 *>(row + my.u0) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
                *reinterpret_cast<uint2 *>(row + my.u0 + my.du) = make_uint2(p[4] | p[5] << 16, p[6] | p[7] << 16);
            };
            float2 w[P::kW];
            my.angles(cs, r, w);
            my.turn(kx, ky, k_row(r, h), cs, r, w, f);
            store(a.k_cache + at, inv[run][2 * own]);
            Elem<T>::unpack(vx, f);
            Elem<T>::unpack(vy, f + 8);
            store(a.v_cache + at, inv[run][2 * own + 1]);
        }

        // ---- the rows that a block held before, where its scale grew
        for (int task = tid >> 5; grown[turn_of] && task < runs * 2 * kHeads; task += kThreads8 / 32) {
            const int run = task / (2 * kHeads), which = task & 1, o = (task >> 1) % kHeads;
            const int64_t slot = slot_of(run_row[run]);
            if (slot < 0 || hb + o >= h_end) continue;
            const float s = ratio[run][task % (2 * kHeads)];
            if (s == 1.f) continue;
            const int off = run_off[run];
            uint8_t *block = (which ? a.v_cache : a.k_cache) + ((size_t)(slot >> lb) * a.Hkv + hb + o) * a.B * D;
            // a lane's 16 codes of every 512, four loads in flight (a block has at most 4096)
            for (int i0 = lane * 16; i0 < off * D; i0 += 2048) {
                uint4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4 *>(block + min(i0 + 512 * i, off * D - 16));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    auto again = [&](uint32_t x) {
                        const float2 lo = values2(x & 0xffffu), hi = values2(x >> 16);
                        return codes2(lo.x * s, lo.y * s) | codes2(hi.x * s, hi.y * s) << 16;
                    };
                    if (i0 + 512 * i < off * D)
                        *reinterpret_cast<uint4 *>(block + i0 + 512 * i) = make_uint4(again(w[i].x), again(w[i].y), again(w[i].z), again(w[i].w));
                }
            }
        }
        kx = kx1, ky = ky1, vx = vx1, vy = vy1;
    }
}

template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D>
cudaError_t launch_write8_t(const Write8Args &a, cudaStream_t st) {
    // CTAs enough for the card where the work allows: KV heads each in CTAs of their own for a step, two CTAs a
    // tile and more heads each for a prompt (the angles of a tile then serve them all); the same for the queries' heads
    constexpr int kHeads = kThreads8 / (kTile * (D / 16)), kRound = kThreads8 / (D / 16);
    const int tiles = (a.T + kTile - 1) / kTile, steps = (a.Hkv + kHeads - 1) / kHeads;
    int kv_parts = (4 * 152 + tiles - 1) / tiles;
    kv_parts = kv_parts < steps ? kv_parts : steps;
    const int pairs = a.q ? (a.T + 1) / 2 : 0, rounds = a.q ? (2 * a.Hq + kRound - 1) / kRound : 1;
    int q_parts = pairs ? (4 * 152 + pairs - 1) / pairs : 1;
    q_parts = q_parts < rounds ? q_parts : rounds;
    const long long ctas = (long long)tiles * kv_parts + (long long)pairs * q_parts;
    if (ctas > 0x7fffffffLL) return cudaErrorNotSupported;
    const dim3 grid((unsigned)ctas);
    const size_t smem = a.R ? (size_t)(kTile + a.B) * (D / 2 + 8) * sizeof(float2) : 0;  // at most 27 KB
    if (a.R == 0 || a.interleaved) return launch_dependent(write8_kernel<T, D, kNeighbours>, grid, kThreads8, smem, st, a, kv_parts, q_parts);
    if (a.R % 16 == 0) return launch_dependent(write8_kernel<T, D, kHalves>, grid, kThreads8, smem, st, a, kv_parts, q_parts);
    return launch_dependent(write8_kernel<T, D, kSplit>, grid, kThreads8, smem, st, a, kv_parts, q_parts);
}

// grid (pairs, K and V): a block's codes in 16-byte units, and its scales.
// (One load and one store in flight a thread: 64 blocks of 8 heads, B 16, D 128 take 3.3 us, 1000 of them 16 for a floor
// of 9.7, 4 blocks of 32 heads and B 32 12.7.  pa_copy_blocks takes 2.3, 21.6 and 2.2 for twice the bytes.)
__global__ void __launch_bounds__(kThreads8) copy_blocks8_kernel(uint8_t *k, uint8_t *v, float *ks, float *vs, const int64_t *pairs,
                                                                 int N, int64_t block_bytes, int Hkv, unsigned int *err) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t src = pairs[2 * blockIdx.x], dst = pairs[2 * blockIdx.x + 1];
    if (src < 0 || src >= N || dst < 0 || dst >= N) {
        if (threadIdx.x == 0) set_error(err, PA_DEVERR_BAD_PAIR);
        return;
    }
    uint8_t *codes = blockIdx.y ? v : k;
    float *scales = blockIdx.y ? vs : ks;
    const uint4 *from = reinterpret_cast<const uint4 *>(codes + src * block_bytes);
    uint4 *to = reinterpret_cast<uint4 *>(codes + dst * block_bytes);
    for (int64_t i = threadIdx.x; i < block_bytes / 16; i += kThreads8) to[i] = from[i];
    for (int h = threadIdx.x; h < Hkv; h += kThreads8) scales[dst * Hkv + h] = scales[src * Hkv + h];
}

}  // namespace

cudaError_t launch_write8(const Write8Args &a, bool bf16, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    if (a.D == 64) return bf16 ? launch_write8_t<__nv_bfloat16, 64>(a, st) : launch_write8_t<__half, 64>(a, st);
    if (a.D == 128) return bf16 ? launch_write8_t<__nv_bfloat16, 128>(a, st) : launch_write8_t<__half, 128>(a, st);
    return cudaErrorNotSupported;
}

cudaError_t launch_copy_blocks8(uint8_t *k, uint8_t *v, float *ks, float *vs, const int64_t *pairs, int P, int N,
                                int64_t block_bytes, int Hkv, unsigned int *err, cudaStream_t st) {
    if (P == 0) return cudaSuccess;
    return launch_dependent(copy_blocks8_kernel, dim3((unsigned)P, 2u), kThreads8, 0, st, k, v, ks, vs, pairs, N, block_bytes, Hkv, err);
}

}  // namespace pa
