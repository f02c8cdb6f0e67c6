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
// Work.  The tokens of one block stand next to each other in the list (a run).  A CTA takes the runs that start
// among its tile of 16 tokens, for one KV head (two at D 64) with its query heads, so a block's scale has one writer.
// Sixteen rows of keys and values stay in registers from the maxima, through the scales, to the codes; further rows
// (runs may begin anywhere in a tile) are read again.  The queries of the same rows are turned while the scales
// settle, and all first loads are under way before the angles are computed (as in pa_rope.cuh, once per (row, pair) in
// shared memory).  Rows that a block held before are rescaled by the same CTA where the scale grew.
//
// Bound: HBM for a prompt (each q element read and written, each k, v element read as 16 bits and written
// as 8), latency for a step.
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

template <typename T, int D, int kPairing>
__global__ void __launch_bounds__(kThreads8) write8_kernel(const Write8Args a) {
    constexpr int L = D / 16;                 // lanes of a row: two units of 8 elements each
    constexpr int kHeads = 128 / (kTile * L);  // KV heads of a CTA: 1 (D 128) or 2
    constexpr int kQ = 4;                     // query heads in flight
    // [rows][kRow]: a row's (cos, sin), those that one thread needs kCols apart, rows off each other by some banks
    constexpr int kA = kPairing == kHalves ? 8 : kPairing == kNeighbours ? 4 : 1;   // pairs of a unit
    constexpr int kCols = D / 2 / kA, kRow = D / 2 + 8;
    extern __shared__ float2 cs[];
    __shared__ unsigned long long fractions[D / 2];   // of a turn, per pair: fp64 work, once a CTA
    __shared__ int64_t slots[kRows + 2];
    __shared__ uint32_t top[2][kHeads][kRows];   // loudest value of each row (bits)
    __shared__ float inv[2][kHeads][kRows];      // per run: 1 / scale
    __shared__ float ratio[2][kHeads][kRows];    // per run: old scale / new where the block's earlier rows change, else 1
    const int tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the runs that start in the tile: slots[j] is token t0 + j - 1
    const int t0 = blockIdx.x * kTile, span = kTile + a.B, half = a.R / 2;
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

    // ---- a thread's row of a pass, its KV head and its two units of a head
    const int prow = tid / L % kTile, own = tid / (kTile * L), c = tid % L;
    const bool live_head = blockIdx.y * kHeads + own < a.Hkv;
    const int h = min((int)blockIdx.y * kHeads + own, a.Hkv - 1);   // KV head
    const int turning = half / 8;
    const bool turns = kPairing != kHalves || c < turning;  // kHalves: whether the units are a pair that turns
    const int u0 = kPairing == kHalves ? (turns ? 8 * c : a.R + 8 * (c - turning)) : 8 * c;
    const int du = kPairing == kHalves ? (turns ? half : (D - a.R) / 2) : D / 2;
    auto load = [&](const T *head, uint4 &x, uint4 &y) {
        x = *reinterpret_cast<const uint4 *>(head + u0);
        y = *reinterpret_cast<const uint4 *>(head + u0 + du);
    };
    auto k_row = [&](int r) { return static_cast<const T *>(a.k) + (size_t)(tok0 + r) * a.k_stride + (size_t)h * D; };
    auto v_row = [&](int r) { return static_cast<const T *>(a.v) + (size_t)(tok0 + r) * a.v_stride + (size_t)h * D; };
    const int G = a.q ? a.Hq / a.Hkv : 0;
    auto q_row = [&](int r, int n) { return static_cast<const T *>(a.q) + (size_t)(tok0 + r) * a.q_stride + ((size_t)h * G + n) * D; };

    // ---- the first pass's loads
    // (threads past the rows or heads load what others do, so that nothing branches around a load)
    uint4 kx, ky, vx, vy, qx[kQ], qy[kQ];
    float old_scale = 0.f;   // of K in lane 0 of a run's first row, of V in lane 1
    {
        const int r = min(prow, rows - 1);
        load(k_row(r), kx, ky);
        load(v_row(r), vx, vy);
#pragma unroll
        for (int n = 0; n < kQ; ++n)
            if (n < G) load(q_row(r, n), qx[n], qy[n]);
        const int64_t slot = slot_of(r);
        if (c < 2 && slot >= 0) old_scale = (c ? a.v_scales : a.k_scales)[(size_t)(slot >> lb) * a.Hkv + h];
    }
    for (int e = tid; e < rows * half; e += kThreads8) {
        const int r = e / half, p = e - r * half;
        cs[r * kRow + p % kA * kCols + p / kA] = turn_at(fractions[p], pair_position(a, tok0 + r, p), a.mscale);
    }

    // ---- the loudest value of each row and head
    auto loudest_of_row = [&](const uint4 &x, const uint4 &y) {
        uint32_t m = loudest<T>(x, y);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    };
    for (int r = prow; r < (rows + kTile - 1) / kTile * kTile; r += kTile) {
        uint4 x = kx, y = ky, z = vx, w = vy;
        const bool here = r < rows && live_head;
        if (r >= kTile && here) {
            load(k_row(r), x, y);
            load(v_row(r), z, w);
        }
        const uint32_t mk = loudest_of_row(x, y), mv = loudest_of_row(z, w);
        if (c == 0 && here) {
            top[0][own][r] = mk;
            top[1][own][r] = mv;
        }
    }
    __syncthreads();

    // ---- the scales of each run: lane 0 of its first row for K, lane 1 for V
    for (int r = prow; r < rows; r += kTile) {
        const int64_t slot = slot_of(r);
        if (c >= 2 || !live_head || slot < 0 || !begins(r)) continue;
        uint32_t m = top[c][own][r];
        int off = (int)(slot & (a.B - 1));
        for (int n = r + 1; n < rows && !begins(n); ++n) {
            m = max(m, top[c][own][n]);
            off = min(off, (int)(slot_of(n) & (a.B - 1)));
        }
        const float x = Bits16<T>::value(m);
        float *at = (c ? a.v_scales : a.k_scales) + (size_t)(slot >> lb) * a.Hkv + h;
        float s = c || half == 0 ? scale_of(x, kLoudestPlain) : scale_of(x * fmaxf(1.f, fabsf(a.mscale)), kLoudestTurned);
        float grew = 1.f;
        if (off > 0) {
            const float old = r < kTile ? old_scale : *at;
            if (old < s) grew = old / s;
            else s = fmaxf(old, s);  // an old scale that is no number counts as none
        }
        *at = s;
        const int run = run_of(r);
        inv[c][own][run] = 1.f / s;
        ratio[c][own][run] = grew;
    }

    // f: the 16 values of a head that this thread has, turned by w, its pairs' (cos, sin).  (x, y) are its units, `head`
    // where they come from.
    constexpr int kW = kPairing == kSplit ? 1 : 8;
    auto angles = [&](int r, float2 (&w)[kW]) {
        if (half == 0) return;  // nothing turns, and no angles were computed
        if constexpr (kPairing == kHalves) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = cs[r * kRow + e * kCols + (turns ? c : 0)];
        } else if constexpr (kPairing == kNeighbours) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = cs[r * kRow + (e & 3) * kCols + (e < 4 ? c : c + L)];
        }
    };
    auto turn = [&](const uint4 &x, const uint4 &y, const T *head, int r, const float2 (&w)[kW], float (&f)[16]) {
        Elem<T>::unpack(x, f);
        Elem<T>::unpack(y, f + 8);
        if constexpr (kPairing == kHalves) {
            if (turns) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = f[e] * w[e].x - f[8 + e] * w[e].y;
                    f[8 + e] = f[8 + e] * w[e].x + f[e] * w[e].y;
                    f[e] = p;
                }
            }
        } else if constexpr (kPairing == kNeighbours) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int p = (e < 4 ? u0 : u0 + du) / 2 + (e & 3);
                if (p < half) {
                    const float v = f[2 * e] * w[e].x - f[2 * e + 1] * w[e].y;
                    f[2 * e + 1] = f[2 * e + 1] * w[e].x + f[2 * e] * w[e].y;
                    f[2 * e] = v;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int d = (e < 8 ? u0 : u0 + du) + (e & 7);
                if (d < a.R) {
                    const bool low = d < half;
                    const float2 t = cs[r * kRow + (low ? d : d - half)];
                    const float other = static_cast<float>(head[low ? d + half : d - half]);
                    f[e] = low ? f[e] * t.x - other * t.y : f[e] * t.x + other * t.y;
                }
            }
        }
    };

    // ---- queries, while the scales settle
    for (int r = prow; r < (rows + kTile - 1) / kTile * kTile; r += kTile) {
        const bool here = r < rows && live_head && slot_of(r < rows ? r : 0) >= 0;
        float2 w[kW];
        if (here) angles(r, w);
        for (int n0 = 0; n0 < G; n0 += kQ) {
            if (here) {
                if (r >= kTile || n0 > 0) {
#pragma unroll
                    for (int n = 0; n < kQ; ++n)
                        if (n0 + n < G) load(q_row(r, n0 + n), qx[n], qy[n]);
                }
#pragma unroll
                for (int n = 0; n < kQ; ++n) {
                    if (n0 + n >= G) break;
                    float f[16];
                    turn(qx[n], qy[n], q_row(r, n0 + n), r, w, f);
                    qx[n] = make_uint4(Mma16<T>::pack(f[0], f[1]), Mma16<T>::pack(f[2], f[3]), Mma16<T>::pack(f[4], f[5]), Mma16<T>::pack(f[6], f[7]));
                    qy[n] = make_uint4(Mma16<T>::pack(f[8], f[9]), Mma16<T>::pack(f[10], f[11]), Mma16<T>::pack(f[12], f[13]), Mma16<T>::pack(f[14], f[15]));
                }
            }
            __syncwarp();  // q_out may be q: the lanes of a row have read it
            if (here) {
                T *to = static_cast<T *>(a.q_out) + (size_t)(tok0 + r) * a.q_out_stride + ((size_t)h * G + n0) * D + u0;
#pragma unroll
                for (int n = 0; n < kQ; ++n)
                    if (n0 + n < G) {
                        *reinterpret_cast<uint4 *>(to + n * D) = qx[n];
                        *reinterpret_cast<uint4 *>(to + n * D + du) = qy[n];
                    }
            }
        }
    }
    __syncthreads();

    // ---- keys and values
    for (int r = prow; r < rows && live_head; r += kTile) {
        const int64_t slot = slot_of(r);
        if (slot < 0) continue;
        if (r >= kTile) {
            load(k_row(r), kx, ky);
            load(v_row(r), vx, vy);
        }
        const int run = run_of(r);
        const size_t at = (((size_t)(slot >> lb) * a.Hkv + h) * a.B + (size_t)(slot & (a.B - 1))) * D;
        float f[16];
        auto store = [&](uint8_t *row, float s) {
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = codes2(f[2 * e] * s, f[2 * e + 1] * s);
            *reinterpret_cast<uint2 *>(row + u0) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
            *reinterpret_cast<uint2 *>(row + u0 + du) = make_uint2(p[4] | p[5] << 16, p[6] | p[7] << 16);
        };
        float2 w[kW];
        angles(r, w);
        turn(kx, ky, k_row(r), r, w, f);
        store(a.k_cache + at, inv[0][own][run]);
        Elem<T>::unpack(vx, f);
        Elem<T>::unpack(vy, f + 8);
        store(a.v_cache + at, inv[1][own][run]);
    }

    // ---- the rows that a block held before, where its scale grew
    for (int task = tid >> 5; task < rows * 2 * kHeads; task += kThreads8 / 32) {
        const int r = task % rows, which = task / rows & 1, o = task / (2 * rows);
        const int64_t slot = slot_of(r);
        if (!begins(r) || slot < 0 || blockIdx.y * kHeads + o >= a.Hkv) continue;
        const float s = ratio[which][o][run_of(r)];
        if (s == 1.f) continue;
        int off = (int)(slot & (a.B - 1));
        for (int n = r + 1; n < rows && !begins(n); ++n) off = min(off, (int)(slot_of(n) & (a.B - 1)));
        uint8_t *block = (which ? a.v_cache : a.k_cache) + ((size_t)(slot >> lb) * a.Hkv + blockIdx.y * kHeads + o) * a.B * D;
        for (int i = lane * 4; i < off * D; i += 128) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(block + i);
            const float2 lo = values2(w & 0xffffu), hi = values2(w >> 16);
            *reinterpret_cast<uint32_t *>(block + i) = codes2(lo.x * s, lo.y * s) | codes2(hi.x * s, hi.y * s) << 16;
        }
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
    constexpr int kHeads = 128 / (kTile * (D / 16));
    const dim3 grid((unsigned)((a.T + kTile - 1) / kTile), (unsigned)((a.Hkv + kHeads - 1) / kHeads));
    if (grid.y > 65535) return cudaErrorNotSupported;
    const size_t smem = a.R ? (size_t)(kTile + a.B) * (D / 2 + 8) * sizeof(float2) : 0;  // at most 27 KB
    if (a.R == 0 || a.interleaved) return launch_dependent(write8_kernel<T, D, kNeighbours>, grid, kThreads8, smem, st, a);
    if (a.R % 16 == 0) return launch_dependent(write8_kernel<T, D, kHalves>, grid, kThreads8, smem, st, a);
    return launch_dependent(write8_kernel<T, D, kSplit>, grid, kThreads8, smem, st, a);
}

// grid (pairs, K and V): a block's codes in 16-byte units, and its scales.
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
