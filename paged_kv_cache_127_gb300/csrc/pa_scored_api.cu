// pa_scored_api.cu -- C-ABI entry points of scored attention, rotary positions
// with the KV write, and eviction: argument validation, workspace sizing, and
// dispatch.  See include/pa.h for the contract of each call.
#include <cmath>
#include <cstdint>

#include "../../include/pa.h"
#include "pa_scored.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int elem_bytes(int dtype) { return dtype == PA_F32 ? 4 : 2; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
bool overlap(const void *p, size_t n, const void *q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n && m && a < b + m && b < a + n;
}
// The same for `rows` rows of `row` bytes, `step` bytes apart, and as many of `wide` bytes, `other` apart:
// rows of one step that lie in each other's gaps (column ranges of one tensor) are apart.
bool rows_overlap(const void *p, int64_t step, int64_t row, const void *q, int64_t other, int64_t wide, int64_t rows) {
    if (!overlap(p, (size_t)((rows - 1) * step + row), q, (size_t)((rows - 1) * other + wide))) return false;
    if (step != other) return true;
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) % step;
    const int64_t gap = off < 0 ? off + step : off;  // from a row of p to the next row of q
    return gap < row || step - gap < wide;
}
int32_t to_status(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    return e == cudaErrorNotSupported ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
}

int32_t check_score(const pa_score *sc) {
    if (!sc) return PA_OK;
    if (!std::isfinite(sc->softcap) || sc->softcap < 0.f || sc->window < 0) return PA_ERR_INVALID;
    if (!aligned(sc->slopes, 4) || !aligned(sc->key_begin, 4) || !aligned(sc->key_end, 4)) return PA_ERR_INVALID;
    return PA_OK;
}

// Rows of key sums: enough columns for every position of the tables.
int32_t check_sums(const pa_key_sums *ks, int64_t cap) {
    if (!ks->sums || !aligned(ks->sums, 16) || !aligned(ks->rows, 4)) return PA_ERR_INVALID;
    if (ks->num_rows < 0 || ks->cols < cap || ks->cols % 4 != 0) return PA_ERR_INVALID;
    return PA_OK;
}

// Scored-attention workspace, each part 256-byte aligned:
//   header    4 ints: work items, claim counter, rows to merge, partition size chosen
//   list      int4 [list_entries]
//   merge     int4 [T]: rows whose range lies in several partitions (only with partials)
//   acc, ml   float [T, Hq, P, D] and [T, Hq, P, 2]   (acc only if P > 1)
//   logits    float [S, Hq, cap]                      (only with sums)
struct ScoredLayout {
    size_t list, merge, acc, ml, logits, total;
};
ScoredLayout scored_layout(const pa_dims *d, size_t list_entries, size_t T, int32_t parts, bool partials, bool sums) {
    ScoredLayout L{};
    size_t off = 256;
    L.list = off;
    off += up256(list_entries * sizeof(int4));
    L.merge = off;
    off += partials ? up256(T * sizeof(int4)) : 0;
    L.acc = off;
    off += partials ? up256(T * d->num_q_heads * parts * d->head_dim * sizeof(float)) : 0;
    L.ml = off;
    off += partials || sums ? up256(T * d->num_q_heads * parts * 2 * sizeof(float)) : 0;
    L.logits = off;
    off += sums ? up256(T * d->num_q_heads * d->max_blocks_per_seq * (size_t)d->block_size * sizeof(float)) : 0;
    L.total = off;
    return L;
}

int32_t check_scored_decode(const pa_dims *d, int32_t *parts) {
    if (!d) return PA_ERR_INVALID;
    const int32_t rc = pa::check_attention(d, pa::decode_partition_size(d), parts);
    if (rc != PA_OK) return rc;
    return (int64_t)d->num_seqs * d->num_q_heads > INT32_MAX ? PA_ERR_INVALID : PA_OK;
}

int32_t check_scored_chunk(const pa_dims *d, int32_t T, int32_t max_q, int32_t *parts) {
    if (!d) return PA_ERR_INVALID;
    const int32_t rc = pa::check_attention(d, pa::chunk_partition_size(d), parts);
    if (rc != PA_OK) return rc;
    if (T < 0 || max_q < 1 || max_q > (1 << 20) || d->num_seqs > 65535) return PA_ERR_INVALID;
    // work items of the plan, at most: row blocks of every sequence (16 rows or more each) x partitions
    const int64_t G = d->num_q_heads / d->num_kv_heads;
    if ((max_q * G / 16 + 1) * d->num_seqs > INT32_MAX / *parts) return PA_ERR_INVALID;
    return (int64_t)T * d->num_q_heads > INT32_MAX ? PA_ERR_INVALID : PA_OK;
}

ScoredLayout decode_layout(const pa_dims *d, int32_t parts, bool sums) {
    return scored_layout(d, (size_t)d->num_seqs * parts, (size_t)d->num_seqs, parts, parts > 1, sums);
}

// f32 chunks have no list; the tcgen05 path has no partials (it walks a tile's whole span).
ScoredLayout chunk_layout(const pa_dims *d, int32_t T, int32_t max_q, int32_t parts) {
    const int G = d->num_q_heads / d->num_kv_heads;
    const bool f32 = d->kv_dtype == PA_F32, umma = !f32 && pa::chunk_uses_umma(max_q, G);
    const int64_t rows = umma ? pa::chunk_umma_rows(max_q, G) : 16 * pa::chunk_row_warps(max_q, G);
    const size_t blocks = (size_t)(((int64_t)max_q * G + rows - 1) / rows) * d->num_seqs;
    return scored_layout(d, f32 ? 0 : blocks * (umma ? 1 : parts), (size_t)T, parts, parts > 1 && !umma, false);
}

void fill_args(pa::ScoredArgs &a, const pa_dims *d, const pa_score *sc, const ScoredLayout &L, void *workspace) {
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.plan_hdr = reinterpret_cast<int *>(ws);
    a.plan_list = reinterpret_cast<int4 *>(ws + L.list);
    a.merge_list = reinterpret_cast<int4 *>(ws + L.merge);
    a.ws_acc = reinterpret_cast<float *>(ws + L.acc);
    a.ws_ml = reinterpret_cast<float *>(ws + L.ml);
    a.S = d->num_seqs;
    a.Hq = d->num_q_heads;
    a.Hkv = d->num_kv_heads;
    a.D = d->head_dim;
    a.B = d->block_size;
    a.N = d->num_blocks;
    a.max_blocks = d->max_blocks_per_seq;
    a.head_group = pa::decode_head_group(d->num_kv_heads);
    if (sc) {
        a.softcap = sc->softcap;
        a.window = sc->window;
        a.slopes = sc->slopes;
        a.key_begin = sc->key_begin;
        a.key_end = sc->key_end;
    }
}

}  // namespace

extern "C" {

size_t pa_decode_scored_workspace_bytes(const pa_dims *dims, int32_t with_sums) {
    int32_t parts = 0;
    if (check_scored_decode(dims, &parts) != PA_OK || dims->num_seqs == 0) return 0;
    return decode_layout(dims, parts, with_sums != 0).total;
}

int32_t pa_decode_scored(const pa_dims *dims, const pa_score *score, const void *q, const void *k_cache,
                         const void *v_cache, const int32_t *block_tables, const int32_t *context_lens, float scale,
                         const pa_key_sums *key_sums, void *out, int32_t out_dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
    int32_t parts = 0;
    int32_t rc = check_scored_decode(dims, &parts);
    if (rc == PA_OK) rc = check_score(score);
    if (rc != PA_OK) return rc;
    if (out_dtype != PA_F32 && out_dtype != dims->kv_dtype) return PA_ERR_INVALID;
    if (key_sums) {
        rc = check_sums(key_sums, (int64_t)dims->max_blocks_per_seq * dims->block_size);
        if (rc != PA_OK) return rc;
    }
    if (dims->num_seqs == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_INVALID;
    const ScoredLayout L = decode_layout(dims, parts, key_sums != nullptr);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)) return PA_ERR_INVALID;

    pa::ScoredArgs a{};
    fill_args(a, dims, score, L, workspace);
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.out = out;
    a.out16 = out_dtype != PA_F32;
    a.scale = scale;
    a.T = dims->num_seqs;
    a.max_query_len = 1;
    a.partition_size = pa::decode_partition_size(dims);
    a.max_parts = parts;
    if (key_sums) {
        a.ws_logits = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + L.logits);
        a.sums = key_sums->sums;
        a.sum_rows = key_sums->rows;
        a.sum_num_rows = key_sums->num_rows;
        a.sum_cols = key_sums->cols;
    }
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf16 = dims->kv_dtype == PA_BF16;
    if (dims->kv_dtype == PA_F32) {
        e = pa::launch_scored_rows(a, st);
    } else {
        // work list, the persistent tensor-core kernel, then merge and sums
        // (each launch a programmatic dependent of the one before)
        const long long block_heads = (long long)dims->num_blocks * dims->num_kv_heads;
        CUtensorMap tmk, tmv;
        e = pa::cached_cache_map(k_cache, bf16, dims->head_dim, dims->block_size, block_heads, a.head_group, &tmk);
        if (e == cudaSuccess)
            e = pa::cached_cache_map(v_cache, bf16, dims->head_dim, dims->block_size, block_heads, a.head_group, &tmv);
        if (e != cudaSuccess) return PA_ERR_CUDA;
        a.listed = 1;
        a.widen = dims->partition_size == 0;
        e = bf16 ? pa::scored_decode_ctas_bf16(a, &a.ctas) : pa::scored_decode_ctas_f16(a, &a.ctas);
        if (e == cudaSuccess) e = pa::launch_scored_decode_plan(a, st);
        if (e == cudaSuccess)
            e = bf16 ? pa::launch_scored_decode_bf16(a, tmk, tmv, st) : pa::launch_scored_decode_f16(a, tmk, tmv, st);
    }
    if (e != cudaSuccess) return to_status(e);
    const bool listed = dims->kv_dtype != PA_F32;
    return to_status(listed && !a.sums ? pa::launch_scored_merge(a, bf16, st)
                                       : pa::launch_scored_finish(a, listed, bf16, st));
}

size_t pa_chunk_scored_workspace_bytes(const pa_dims *dims, int32_t num_tokens, int32_t max_query_len) {
    int32_t parts = 0;
    if (check_scored_chunk(dims, num_tokens, max_query_len, &parts) != PA_OK) return 0;
    return chunk_layout(dims, num_tokens, max_query_len, parts).total;
}

int32_t pa_chunk_scored(const pa_dims *dims, const pa_score *score, const void *q, const void *k_cache,
                        const void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                        const int32_t *query_start, int32_t num_tokens, int32_t max_query_len, float scale, void *out,
                        int32_t out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    int32_t parts = 0;
    int32_t rc = check_scored_chunk(dims, num_tokens, max_query_len, &parts);
    if (rc == PA_OK) rc = check_score(score);
    if (rc != PA_OK) return rc;
    if (out_dtype != PA_F32 && out_dtype != dims->kv_dtype) return PA_ERR_INVALID;
    if (dims->num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !out) return PA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4))
        return PA_ERR_INVALID;
    const ScoredLayout L = chunk_layout(dims, num_tokens, max_query_len, parts);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)) return PA_ERR_INVALID;

    pa::ScoredArgs a{};
    fill_args(a, dims, score, L, workspace);
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.out = out;
    a.out16 = out_dtype != PA_F32;
    a.scale = scale;
    a.T = num_tokens;
    a.max_query_len = max_query_len;
    a.partition_size = pa::chunk_partition_size(dims);
    a.max_parts = parts;
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf16 = dims->kv_dtype == PA_BF16;
    if (dims->kv_dtype == PA_F32) {
        e = pa::launch_scored_rows(a, st);
        if (e != cudaSuccess) return to_status(e);
        return to_status(pa::launch_scored_finish(a, false, false, st));
    }
    const int G = dims->num_q_heads / dims->num_kv_heads;
    const bool umma = pa::chunk_uses_umma(max_query_len, G);
    a.row_warps = pa::chunk_row_warps(max_query_len, G);
    a.umma_rows = umma ? pa::chunk_umma_rows(max_query_len, G) : 0;
    const long long block_heads = (long long)dims->num_blocks * dims->num_kv_heads;
    const int box_heads = umma ? 1 : a.head_group;
    CUtensorMap tmk, tmv;
    e = pa::cached_cache_map(k_cache, bf16, dims->head_dim, dims->block_size, block_heads, box_heads, &tmk);
    if (e == cudaSuccess)
        e = pa::cached_cache_map(v_cache, bf16, dims->head_dim, dims->block_size, block_heads, box_heads, &tmv);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    if (umma) {
        // long chunks: plan, then the tcgen05 kernel, which loads queries and stores full tiles by TMA
        CUtensorMap tmq, tmo;
        e = pa::cached_query_map(q, bf16, dims->head_dim, dims->num_q_heads, num_tokens, G, &tmq);
        if (e == cudaSuccess)
            e = a.out16 ? pa::cached_query_map(out, bf16, dims->head_dim, dims->num_q_heads, num_tokens, G, &tmo)
                        : pa::cached_output_map(static_cast<float *>(out), dims->head_dim, dims->num_q_heads, num_tokens, G,
                                                &tmo);
        if (e != cudaSuccess) return PA_ERR_CUDA;
        e = pa::launch_scored_chunk_plan(a, st);
        if (e == cudaSuccess)
            e = bf16 ? pa::launch_scored_umma_bf16(a, tmk, tmv, tmq, tmo, st)
                     : pa::launch_scored_umma_f16(a, tmk, tmv, tmq, tmo, st);
        return to_status(e);
    }
    // short chunks: plan, the mma.sync kernel, merge
    e = pa::launch_scored_chunk_plan(a, st);
    if (e == cudaSuccess)
        e = bf16 ? pa::launch_scored_chunk_bf16(a, tmk, tmv, st) : pa::launch_scored_chunk_f16(a, tmk, tmv, st);
    if (e != cudaSuccess) return to_status(e);
    return to_status(pa::launch_scored_merge(a, bf16, st));
}

int32_t pa_rope_write_kv(const pa_dims *dims, const pa_rope *rope, const void *q, int64_t q_stride, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                         const int64_t *slot_mapping, int32_t num_tokens, void *q_out, int64_t q_out_stride,
                         void *k_cache, void *v_cache, void *stream) {
    const int32_t rc = pa::check_cache(dims);
    if (rc != PA_OK) return rc;
    if (!rope || num_tokens < 0) return PA_ERR_INVALID;
    if (dims->num_q_heads <= 0 || dims->num_q_heads % dims->num_kv_heads != 0) return PA_ERR_INVALID;
    if (rope->rotary_dim < 2 || rope->rotary_dim > dims->head_dim || rope->rotary_dim % 2 != 0 ||
        (rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->mscale))
        return PA_ERR_INVALID;
    const int64_t es = elem_bytes(dims->kv_dtype);
    const int64_t q_row = (int64_t)dims->num_q_heads * dims->head_dim, kv_row = (int64_t)dims->num_kv_heads * dims->head_dim;
    if (q_row > INT32_MAX / 4) return PA_ERR_INVALID;
    if ((int64_t)dims->block_size * dims->head_dim > INT32_MAX) return PA_ERR_INVALID;  // a head's rows of a block, in 32 bits
    if (num_tokens == 0) return PA_OK;
    if (!rope->freqs || !q || !k || !v || !positions || !slot_mapping || !q_out || !k_cache || !v_cache)
        return PA_ERR_INVALID;
    if (q_stride < q_row || q_out_stride < q_row || k_stride < kv_row || v_stride < kv_row) return PA_ERR_INVALID;
    if (q_stride * es % 16 || q_out_stride * es % 16 || k_stride * es % 16 || v_stride * es % 16) return PA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(rope->freqs, 8))
        return PA_ERR_INVALID;
    // q_out is q itself, or apart from it (a token's row is read by other CTAs than the one that writes it)
    if (!(q == q_out && q_stride == q_out_stride) &&
        rows_overlap(q_out, q_out_stride * es, q_row * es, q, q_stride * es, q_row * es, num_tokens))
        return PA_ERR_INVALID;
    if (rows_overlap(q_out, q_out_stride * es, q_row * es, k, k_stride * es, kv_row * es, num_tokens) ||
        rows_overlap(q_out, q_out_stride * es, q_row * es, v, v_stride * es, kv_row * es, num_tokens))
        return PA_ERR_INVALID;
    pa::RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.slots = slot_mapping;
    a.freqs = rope->freqs;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.T = num_tokens;
    a.Hq = dims->num_q_heads;
    a.Hkv = dims->num_kv_heads;
    a.D = dims->head_dim;
    a.R = rope->rotary_dim;
    a.B = dims->block_size;
    a.N = dims->num_blocks;
    a.interleaved = rope->interleaved;
    a.mscale = rope->mscale;
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    return to_status(pa::launch_rope_write_kv(a, dims->kv_dtype, static_cast<cudaStream_t>(stream)));
}

int32_t pa_rope_freqs(int32_t rotary_dim, double theta, int32_t scaling, double factor, double original_len,
                      double fast, double slow, double *freqs_out, float *mscale) {
    const double two_pi = 6.283185307179586476925;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || !freqs_out || !mscale || !std::isfinite(theta) || theta <= 1.0)
        return PA_ERR_INVALID;
    if (scaling < PA_ROPE_PLAIN || scaling > PA_ROPE_BANDS) return PA_ERR_INVALID;
    if (scaling != PA_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return PA_ERR_INVALID;
    const bool banded = scaling == PA_ROPE_RAMP || scaling == PA_ROPE_BANDS;
    if (banded && !(std::isfinite(original_len) && original_len > 0.0 && slow > 0.0 && fast > slow && std::isfinite(fast)))
        return PA_ERR_INVALID;
    if (scaling == PA_ROPE_BASE && rotary_dim <= 2) return PA_ERR_INVALID;
    const double R = rotary_dim;
    if (scaling == PA_ROPE_BASE) theta *= std::pow(factor, R / (R - 2.0));
    // PA_ROPE_RAMP: the pairs between which the ramp runs
    double low = 0.0, high = 0.0;
    if (scaling == PA_ROPE_RAMP) {
        low = std::fmax(0.0, std::floor(R * std::log(original_len / (fast * two_pi)) / (2.0 * std::log(theta))));
        high = std::fmin(R - 1.0, std::ceil(R * std::log(original_len / (slow * two_pi)) / (2.0 * std::log(theta))));
    }
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / R);
        double y = f;
        if (scaling == PA_ROPE_LINEAR) {
            y = f / factor;
        } else if (scaling == PA_ROPE_RAMP) {
            double u = (i - low) / (high > low ? high - low : 1e-3);
            u = u < 0.0 ? 0.0 : (u > 1.0 ? 1.0 : u);
            y = f * (1.0 - u) + f / factor * u;
        } else if (scaling == PA_ROPE_BANDS) {
            const double turns = original_len * f / two_pi;
            double u = (turns - slow) / (fast - slow);
            u = u < 0.0 ? 0.0 : (u > 1.0 ? 1.0 : u);
            y = (1.0 - u) * f / factor + u * f;
        }
        freqs_out[i] = y;
    }
    *mscale = scaling == PA_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return PA_OK;
}

static int32_t check_evict_dims(const pa_dims *d) {
    const int32_t rc = pa::check_cache(d);
    if (rc != PA_OK) return rc;
    if (d->num_seqs < 0 || d->max_blocks_per_seq <= 0) return PA_ERR_INVALID;
    if ((int64_t)d->max_blocks_per_seq * d->block_size > 1 << 30) return PA_ERR_INVALID;  // loops step past it in 32 bits
    if ((int64_t)d->num_seqs * d->num_kv_heads > 65535) return PA_ERR_INVALID;  // the copy grid's y extent
    // cache rows (N * Hkv * B) are numbered in 32 bits
    if ((int64_t)d->num_blocks * d->num_kv_heads > INT32_MAX / d->block_size) return PA_ERR_INVALID;
    return PA_OK;
}

size_t pa_evict_workspace_bytes(const pa_dims *dims) {
    if (check_evict_dims(dims) != PA_OK || dims->num_seqs == 0) return 0;
    const size_t heads = (size_t)dims->num_seqs * dims->num_kv_heads;
    return up256(heads * sizeof(int32_t)) +
           up256(heads * dims->max_blocks_per_seq * (size_t)dims->block_size * sizeof(int32_t));
}

int32_t pa_evict(const pa_dims *dims, void *k_cache, void *v_cache, const int32_t *block_tables,
                 const int32_t *context_lens, const int32_t *new_tables, const int32_t *keep_lens, int32_t recent,
                 const pa_key_sums *key_sums, float *sums_out, int32_t *new_lens, void *workspace,
                 size_t workspace_bytes, void *stream) {
    int32_t rc = check_evict_dims(dims);
    if (rc != PA_OK) return rc;
    if (recent < 0 || !key_sums) return PA_ERR_INVALID;
    rc = check_sums(key_sums, (int64_t)dims->max_blocks_per_seq * dims->block_size);
    if (rc != PA_OK) return rc;
    if (key_sums->cols > 1 << 30) return PA_ERR_INVALID;  // rows are walked in 32-bit steps
    if (dims->num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !new_tables || !keep_lens || !sums_out || !new_lens)
        return PA_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(sums_out, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(new_tables, 4) || !aligned(keep_lens, 4) || !aligned(new_lens, 4))
        return PA_ERR_INVALID;
    const size_t sum_bytes = (size_t)key_sums->num_rows * dims->num_kv_heads * key_sums->cols * sizeof(float);
    if (sums_out != key_sums->sums && overlap(sums_out, sum_bytes, key_sums->sums, sum_bytes)) return PA_ERR_INVALID;
    const size_t len_bytes = (size_t)dims->num_seqs * sizeof(int32_t);
    if (overlap(new_lens, len_bytes, context_lens, len_bytes) || overlap(new_lens, len_bytes, keep_lens, len_bytes))
        return PA_ERR_INVALID;
    if (!workspace || workspace_bytes < pa_evict_workspace_bytes(dims) || !aligned(workspace, 256)) return PA_ERR_INVALID;
    const size_t heads = (size_t)dims->num_seqs * dims->num_kv_heads;
    pa::EvictArgs a{};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.tables = block_tables;
    a.lens = context_lens;
    a.new_tables = new_tables;
    a.keep_lens = keep_lens;
    a.sums = key_sums->sums;
    a.sum_rows = key_sums->rows;
    a.sum_num_rows = key_sums->num_rows;
    a.sum_cols = key_sums->cols;
    a.sums_out = sums_out;
    a.new_lens = new_lens;
    a.counts = static_cast<int32_t *>(workspace);
    a.list = reinterpret_cast<int32_t *>(static_cast<unsigned char *>(workspace) + up256(heads * sizeof(int32_t)));
    a.S = dims->num_seqs;
    a.Hkv = dims->num_kv_heads;
    a.row_bytes = dims->head_dim * elem_bytes(dims->kv_dtype);
    a.B = dims->block_size;
    a.N = dims->num_blocks;
    a.max_blocks = dims->max_blocks_per_seq;
    a.recent = recent;
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    return to_status(pa::launch_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
