// pa_scored.h -- host-side interface of the scored attention, rotary and
// eviction kernels: what their entry points (pa_scored_api.cu) hand to the
// translation units, and the parts of pa_api.cu they share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace pa {

// ------------------------------------------------------------------ shared with pa_api.cu
unsigned int *device_error_word();
int32_t check_cache(const pa_dims *d);
// The decode checks for partitions of `partition` tokens; fills max_parts.
int32_t check_attention(const pa_dims *d, int32_t partition, int32_t *max_parts);
int32_t decode_partition_size(const pa_dims *d);
int32_t chunk_partition_size(const pa_dims *d);
cudaError_t cached_cache_map(const void *ptr, bool bf16, int D, int B, long long block_heads, int hg, CUtensorMap *out);
cudaError_t cached_query_map(const void *q, bool bf16, int D, int Hq, long long T, int G, CUtensorMap *out);
cudaError_t cached_output_map(float *o, int D, int Hq, long long T, int G, CUtensorMap *out);

// ------------------------------------------------------------------ scored attention
// A launch of scored attention, already validated.  A decode is the case of one
// row per sequence: query_start is null, T = S and row s is sequence s.
struct ScoredArgs {
    const void *q;                // [T, Hq, D]
    const void *k_cache;
    const void *v_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_start;   // [S + 1], or null for a decode
    void *out;                    // [T, Hq, D], f32 or the cache's type
    float *ws_ml;                 // [T, Hq, P, 2]  (m in log2 units, l)
    float *ws_acc;                // [T, Hq, P, D]
    float *ws_logits;             // [S, Hq, cap] logits in log2 units; null without sums
    int *plan_hdr;                // [0] work items, [1] claim counter, [2] rows to merge, [3] the
                                  // decode plan's partition size
    int4 *plan_list;              // work items
    int4 *merge_list;             // (row, first partition, last partition, -) of the rows to merge
    unsigned int *err;
    float *sums;                  // [sum_num_rows, Hkv, sum_cols], or null
    const int32_t *sum_rows;      // [S], or null: row s
    const float *slopes;          // [Hq], or null
    const int32_t *key_begin;     // [T], or null
    const int32_t *key_end;       // [T], or null
    int sum_num_rows, sum_cols;
    int S, T, Hq, Hkv, D, B, N, max_blocks, partition_size, max_parts, max_query_len;
    int window;                   // 0: none
    int out16;                    // out is in the cache's 16-bit type
    int head_group;               // KV heads per tensor-core work item
    int row_warps;                // mma.sync chunk path: 16-row tiles per KV head per item
    int umma_rows;                // tcgen05 chunk path: query rows per CTA, else 0
    int ctas;                     // persistent grid of the tensor-core decode
    int listed;                   // decode with a plan: pieces as the plan chose them
    int widen;                    // the plan may choose a multiple of partition_size
    float scale, softcap;         // softcap 0: none
};

// Mark of a work item that holds its sequence's whole range (in the partition's int).
constexpr int kWholeRange = 1 << 30;
// Mark of a tcgen05 chunk item whose rows' ranges may leave keys between them that no row sees (in the
// sequence's int).
constexpr int kHoles = 1 << 30;

// Tensor-core decode (f16 / bf16): the work list, the persistent kernel, and the
// CTAs it launches on the current device (SMs x resident CTAs per SM).
cudaError_t launch_scored_decode_plan(const ScoredArgs &a, cudaStream_t st);
cudaError_t launch_scored_decode_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t launch_scored_decode_bf16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t scored_decode_ctas_f16(const ScoredArgs &a, int *ctas);
cudaError_t scored_decode_ctas_bf16(const ScoredArgs &a, int *ctas);

// Tensor-core chunk attention: the work list, the mma.sync kernel for short chunks
// and the tcgen05 kernel for long ones (tmo: the output's map, 16-bit or f32).
cudaError_t launch_scored_chunk_plan(const ScoredArgs &a, cudaStream_t st);
cudaError_t launch_scored_chunk_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t launch_scored_chunk_bf16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st);
cudaError_t launch_scored_umma_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                   const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st);
cudaError_t launch_scored_umma_bf16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st);

// Merge of the split-K partials of the rows that the plan listed.
cudaError_t launch_scored_merge(const ScoredArgs &a, bool bf16, cudaStream_t st);
// The same without a list (f32 caches: listed false), and with the sums of attention weights.
cudaError_t launch_scored_finish(const ScoredArgs &a, bool listed, bool bf16, cudaStream_t st);
// CUDA-core kernel, one CTA per (row, KV head, partition): f32 caches.
cudaError_t launch_scored_rows(const ScoredArgs &a, cudaStream_t st);

// ------------------------------------------------------------------ rotary positions and KV write
struct RopeArgs {
    const void *q, *k, *v;
    const int32_t *positions;
    const int64_t *slots;
    const double *freqs;
    void *q_out, *k_cache, *v_cache;
    unsigned int *err;
    long long q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
    int T, Hq, Hkv, D, R, B, N, interleaved;
    float mscale;
};
cudaError_t launch_rope_write_kv(const RopeArgs &a, int dtype, cudaStream_t st);

// ------------------------------------------------------------------ eviction
struct EvictArgs {
    void *k_cache, *v_cache;
    const int32_t *tables, *lens, *new_tables, *keep_lens;
    const float *sums;
    const int32_t *sum_rows;
    float *sums_out;
    int32_t *new_lens;
    int32_t *counts;   // [S, Hkv]: rows to move (0: the sequence stays)
    int32_t *list;     // [S, Hkv, cap]: old position of each new one
    unsigned int *err;
    int sum_num_rows, sum_cols;
    int S, Hkv, row_bytes, B, N, max_blocks, recent;
};
cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st);

}  // namespace pa
