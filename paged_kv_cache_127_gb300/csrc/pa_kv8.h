// pa_kv8.h -- host-side interface of the 8-bit cache's kernels: what their entry
// points (pa_kv8_api.cu) hand to the translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace pa {

// Scales are powers of two from 2^kScaleFloor on.  kLoudestPlain times its scale is the largest value of a
// block's codes; a pair that a rotation turns grows by sqrt(2) at most, and 316 sqrt(2) < 448.
constexpr int kScaleFloor = -40;
constexpr float kLoudestPlain = 448.f, kLoudestTurned = 316.f;

// ------------------------------------------------------------------ the write
struct Write8Args {
    const void *q, *k, *v;          // q null: keys and values only
    const int32_t *positions;       // [num_axes, T]
    const int32_t *pair_axis;       // [R / 2], or null: one axis
    const int64_t *slots;
    const double *freqs;
    void *q_out;
    uint8_t *k_cache, *v_cache;
    float *k_scales, *v_scales;
    unsigned int *err;
    long long q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
    int T, Hq, Hkv, D, R, B, N, num_axes, interleaved;
    float mscale;
};
cudaError_t launch_write8(const Write8Args &a, bool bf16, cudaStream_t st);
cudaError_t launch_copy_blocks8(uint8_t *k, uint8_t *v, float *ks, float *vs, const int64_t *pairs, int P, int N,
                                int64_t block_bytes, int Hkv, unsigned int *err, cudaStream_t st);

// ------------------------------------------------------------------ attention
// A decode is the case of one row per sequence: query_start is null, T = S.
struct Attend8Args {
    const void *q;                  // [T, Hq, D]
    const float *k_scales, *v_scales;  // [N, Hkv]
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;     // [S + 1], or null
    void *out;                      // [T, Hq, D], f32 or the queries' type
    int *hdr;                       // [0] whether query_start is in order (mma.sync); work items, claims (tcgen05), or steps of a CTA in [1]
    int4 *list;                     // per (sequence, head group, row block): its first part and their number (int2); tcgen05: work items
    float *parts;                   // mma.sync: two parts of a (row block, head group) per CTA, O and (m, l)
    int4 *notes, *starts;           // tcgen05 line, per CTA: the item it began and others go on with; where it starts
    const uint8_t *k_cache, *v_cache;
    unsigned int *err;
    int groups;                     // tcgen05: row groups of a sequence, at most
    int S, T, Hq, Hkv, D, B, N, max_blocks, max_query_len;
    int window, sinks;              // window 0: none
    int out16;
    int whole;                      // mma.sync path: CTAs take whole (sequence, row block, head group)s
    int units;                      // CTAs, which share the keys (tcgen05: 0: whole items, claimed)
    int tiles;                      // tcgen05 path: 128-row tiles of an item (1 or 2)
    float scale;
};
// mma.sync path, and the join of its parts: `mb` warps with 8 * nq rows each for a row block of a KV head, `hg` KV heads
// a CTA, which has a producer warp besides; up to eight consumers and ten warps an SM.
constexpr int kSms8 = 152;
// tcgen05 line: steps of a CTA at least, where a call has that many (64 tokens over 2000 keys 42 us with 2, 34 with 4, 32 with 8)
constexpr int kLeastSteps8 = 8;
constexpr int attend8_ctas(int nq, int mb, int hg) {   // per SM
    return nq < 3 ? 10 / (hg * mb + 1) : hg * mb == 4 ? 2 : 8 / (hg * mb + 1);
}
struct Rows8 {
    int nq, mb;
};
inline Rows8 attend8_rows(int max_query_len, int G) {
    const long long rows = (long long)max_query_len * G;
    return rows <= 8 ? Rows8{1, 1} : rows <= 16 ? Rows8{1, 2} : rows <= 24 ? Rows8{3, 1} : rows <= 32 ? Rows8{2, 2} : rows <= 48 ? Rows8{3, 2} : Rows8{2, 4};
}
inline int attend8_heads(int Hkv, Rows8 r) {
    return Hkv % 4 == 0 && r.nq * r.mb < 6 ? 4 : Hkv % 2 == 0 ? 2 : 1;
}
cudaError_t launch_attend8_mma_f16_64(const Attend8Args &a, Rows8 rows, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t launch_attend8_mma_f16_128(const Attend8Args &a, Rows8 rows, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t launch_attend8_mma_bf16_64(const Attend8Args &a, Rows8 rows, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t launch_attend8_mma_bf16_128(const Attend8Args &a, Rows8 rows, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
// A cache of codes [N, Hkv, B, D]: boxes of `heads` heads of one block, rows of D bytes with the swizzle of that width.
cudaError_t make_codes_tensor_map(CUtensorMap *map, const void *codes, int D, int B, long long block_heads, int heads);
// tcgen05 path, from 64 rows of a KV head on: the work list, and the kernel (tmq: the queries' map).
cudaError_t launch_attend8_plan(const Attend8Args &a, cudaStream_t st);
cudaError_t launch_attend8_umma_f16(const Attend8Args &a, const CUtensorMap &tmq, cudaStream_t st);
cudaError_t launch_attend8_umma_bf16(const Attend8Args &a, const CUtensorMap &tmq, cudaStream_t st);

}  // namespace pa
