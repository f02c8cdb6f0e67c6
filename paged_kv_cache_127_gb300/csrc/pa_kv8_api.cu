// pa_kv8_api.cu -- C-ABI entry points of the 8-bit cache: argument validation,
// workspace sizing and dispatch.  See include/pa.h for the contract of each call.
#include <cstdint>

#include "../../include/pa.h"
#include "pa_kv8.h"
#include "pa_scored.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
int32_t to_status(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    return e == cudaErrorNotSupported ? PA_ERR_UNSUPPORTED : PA_ERR_CUDA;
}

// What all calls ask of the cache's shape.
int32_t check_shape8(const pa_dims *d) {
    const int32_t rc = pa::check_cache(d);
    if (rc != PA_OK) return rc;
    if (d->kv_dtype == PA_F32 || !(d->head_dim == 64 || d->head_dim == 128) || !(d->block_size == 16 || d->block_size == 32))
        return PA_ERR_UNSUPPORTED;
    // cache rows (N * Hkv * B) are addressed with 32-bit coordinates
    if ((int64_t)d->num_blocks * d->num_kv_heads > INT32_MAX / d->block_size) return PA_ERR_INVALID;
    return PA_OK;
}
int32_t check_cache8(const pa_cache8 *c) {
    if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales) return PA_ERR_INVALID;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4)) return PA_ERR_INVALID;
    return PA_OK;
}

constexpr int32_t kMaxTokens8 = INT32_MAX - 64;   // a write's tokens, and the tile behind the last one, in 32 bits

int32_t check_attend8(const pa_dims *d) {
    const int32_t rc = check_shape8(d);
    if (rc != PA_OK) return rc;
    if (d->num_seqs < 0 || d->num_q_heads <= 0 || d->max_blocks_per_seq <= 0) return PA_ERR_INVALID;
    if (d->num_q_heads % d->num_kv_heads != 0) return PA_ERR_INVALID;
    const int32_t G = d->num_q_heads / d->num_kv_heads;
    if (!(G == 1 || G == 2 || G == 4 || G == 8)) return PA_ERR_UNSUPPORTED;
    // positions, and the step behind the last one, in 32 bits
    if ((int64_t)d->max_blocks_per_seq * d->block_size > INT32_MAX - 4096) return PA_ERR_INVALID;
    if ((int64_t)d->num_seqs * d->num_q_heads > INT32_MAX) return PA_ERR_INVALID;
    return PA_OK;
}
int32_t check_chunk8(const pa_dims *d, int32_t T, int32_t max_q) {
    const int32_t rc = check_attend8(d);
    if (rc != PA_OK) return rc;
    if (T < 0 || max_q < 1 || max_q > (1 << 20) || d->num_seqs > 65535) return PA_ERR_INVALID;
    if ((int64_t)T * d->num_q_heads > INT32_MAX) return PA_ERR_INVALID;
    // the grid of the join: (sequence, KV head, row block of 8 rows or more)
    const int64_t blocks = ((int64_t)max_q * (d->num_q_heads / d->num_kv_heads) + 7) / 8;
    return (int64_t)d->num_seqs * d->num_kv_heads > INT32_MAX / blocks ? PA_ERR_INVALID : PA_OK;
}
int32_t check_window(const pa_window *w) { return w && (w->window < 0 || w->sinks < 0) ? PA_ERR_INVALID : PA_OK; }

constexpr int64_t kWholeKeys8 = 256;

// Workspace, each part 256-byte aligned: a header, the notes of each (sequence, KV head, row block), and two parts
// for each CTA that shares the keys (mma.sync path).
struct Layout8 {
    pa::Rows8 rows;
    int hg, units, whole, tiles, groups;  // tiles 0: the mma.sync path
    size_t list, parts, total;
};
// Keys that the rows of a sequence see, at most.
int64_t reach8(const pa_dims *d, int32_t max_q, const pa_window *w) {
    const int64_t keys = (int64_t)d->max_blocks_per_seq * d->block_size;
    const int64_t seen = w && w->window ? (int64_t)w->window + w->sinks + max_q : keys;
    return seen < keys ? seen : keys;
}
Layout8 layout8(const pa_dims *d, int32_t max_q, const pa_window *w) {
    Layout8 L{};
    const int G = d->num_q_heads / d->num_kv_heads;
    L.rows = pa::attend8_rows(max_q, G);
    L.hg = pa::attend8_heads(d->num_kv_heads, L.rows);
    const int64_t rows = 8 * L.rows.nq * L.rows.mb, blocks = ((int64_t)max_q * G + rows - 1) / rows;
    // no more CTAs than give each of them four steps of 32 keys, or one where 64 CTAs suffice for that
    const int64_t steps = ((int64_t)d->max_blocks_per_seq * d->block_size + 31) / 32;
    const int64_t most = (int64_t)d->num_seqs * (d->num_kv_heads / L.hg) * blocks;  // at most 2^31
    const int64_t cap = pa::kSms8 * pa::attend8_ctas(L.rows.nq, L.rows.mb, L.hg);
    const int64_t all = most > cap * 4 / steps ? cap * 4 : most * steps, fours = (all + 3) / 4;
    const int64_t units = fours > 64 ? fours : (all < 64 ? all : 64);
    L.units = (int)(units < cap ? (units > 0 ? units : 1) : cap);
    L.list = 256;
    L.parts = L.list + up256((size_t)most * sizeof(int2));
    // Up to kWholeKeys8 keys a sequence: whole (sequence, row block, head group)s for each CTA, and no launch that joins parts.
    // (3 sequences of up to 47 keys 8.4 us with equal stretches, 6.3 so; 32 of up to 250 16.2 and 11.7; 256 behind a window
    // of 128 29.8 and 24.6; but 8 behind a window of 512 15.8 and 21.0)
    L.whole = reach8(d, max_q, w) <= kWholeKeys8;
    if (L.whole) {
        L.units = (int)(most < cap ? most : cap);
        L.total = L.parts;
        return L;
    }
    L.total = L.parts + up256((size_t)2 * L.units * L.hg * rows * (d->head_dim + 2) * sizeof(float));
    return L;
}
Layout8 decode_layout8(const pa_dims *d, const pa_window *w) { return layout8(d, 1, w); }
Layout8 chunk_layout8(const pa_dims *d, int32_t max_q, const pa_window *w) {
    const int G = d->num_q_heads / d->num_kv_heads;
    if (!pa::chunk_uses_umma(max_q, G)) return layout8(d, max_q, w);
    Layout8 L{};   // a header and the work list
    L.tiles = pa::chunk_umma_rows(max_q, G) / 128;
    L.list = 256;
    const int64_t groups = ((int64_t)max_q * G + 128 * L.tiles - 1) / (128 * L.tiles);
    L.groups = (int)groups;
    const int64_t items = groups * d->num_seqs * d->num_kv_heads;
    // Fewer items than SMs, with many steps each: all steps in a line that the CTAs share equally (list: notes and starts).
    // That costs some 24 steps' time more (plan, parts, join), and saves a whole item's steps but for the SMs' share.
    // (8 KV heads of 128, by items and with the line: 512 tokens over 30000 keys 475 and 234 us, over 2000 keys 48 and 44;
    // 64 tokens over 2000 keys 40 and 32; a window of 1024 of 64 dimensions 26 and 32, 4 chunks of 512 82 and 87)
    const int64_t steps = (reach8(d, max_q, w) + 63) / 64;
    if (items < pa::kSms8 && steps * (pa::kSms8 - items) > 24 * pa::kSms8) {
        const int64_t units = (items * steps + pa::kLeastSteps8 - 1) / pa::kLeastSteps8;
        L.units = units < pa::kSms8 ? (int)units : pa::kSms8;
        L.parts = L.list + up256((size_t)2 * L.units * sizeof(int4));
        L.total = L.parts + up256((size_t)2 * L.units * 128 * L.tiles * (d->head_dim + 2) * sizeof(float));
        return L;
    }
    L.total = L.list + up256((size_t)(groups * d->num_seqs) * sizeof(int4));
    return L;
}

// The tensor maps of the caches: the last four (caches, shapes) of a host thread.  A model with a cache for each layer
// encodes both maps in every call, which takes 0.1 us (32 caches in turn 3.8 us a prepared decode, one cache 3.7).
cudaError_t codes_map(const void *ptr, int D, int B, long long block_heads, int heads, CUtensorMap *out) {
    struct Entry {
        const void *ptr = nullptr;
        long long block_heads = 0;
        int D = 0, B = 0, heads = 0;
        CUtensorMap map;
    };
    thread_local Entry cache[4];
    thread_local int next = 0;
    for (auto &e : cache)
        if (e.ptr == ptr && e.block_heads == block_heads && e.D == D && e.B == B && e.heads == heads) {
            *out = e.map;
            return cudaSuccess;
        }
    Entry &e = cache[next];
    next = (next + 1) % 4;
    e.ptr = nullptr;
    const cudaError_t rc = pa::make_codes_tensor_map(&e.map, ptr, D, B, block_heads, heads);
    if (rc != cudaSuccess) return rc;
    e.ptr = ptr;
    e.block_heads = block_heads;
    e.D = D;
    e.B = B;
    e.heads = heads;
    *out = e.map;
    return cudaSuccess;
}

void fill8(pa::Attend8Args &a, const pa_dims *d, const pa_window *w, const void *q, const pa_cache8 *c,
           const int32_t *tables, const int32_t *lens, float scale, void *out, int32_t out_dtype, const Layout8 &L, void *workspace) {
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.q = q;
    a.k_cache = static_cast<const uint8_t *>(c->k);
    a.v_cache = static_cast<const uint8_t *>(c->v);
    a.k_scales = c->k_scales;
    a.v_scales = c->v_scales;
    a.block_tables = tables;
    a.context_lens = lens;
    a.out = out;
    a.out16 = out_dtype != PA_F32;
    a.scale = scale;
    a.hdr = reinterpret_cast<int *>(ws);
    a.list = reinterpret_cast<int4 *>(ws + L.list);
    a.parts = reinterpret_cast<float *>(ws + L.parts);
    a.notes = a.list;
    a.starts = a.list + L.units;
    a.units = L.units;
    a.whole = L.whole;
    a.tiles = L.tiles;
    a.groups = L.groups;
    a.S = d->num_seqs;
    a.Hq = d->num_q_heads;
    a.Hkv = d->num_kv_heads;
    a.D = d->head_dim;
    a.B = d->block_size;
    a.N = d->num_blocks;
    a.max_blocks = d->max_blocks_per_seq;
    a.window = w ? w->window : 0;
    a.sinks = w && w->window ? w->sinks : 0;
}

int32_t run_mma(pa::Attend8Args &a, const pa_dims *d, const Layout8 &L, void *stream) {
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    CUtensorMap tmk, tmv;
    const long long block_heads = (long long)a.N * a.Hkv;
    cudaError_t e = codes_map(a.k_cache, a.D, a.B, block_heads, L.hg, &tmk);
    if (e == cudaSuccess) e = codes_map(a.v_cache, a.D, a.B, block_heads, L.hg, &tmv);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d->kv_dtype == PA_BF16)
        e = a.D == 64 ? pa::launch_attend8_mma_bf16_64(a, L.rows, L.hg, tmk, tmv, st) : pa::launch_attend8_mma_bf16_128(a, L.rows, L.hg, tmk, tmv, st);
    else
        e = a.D == 64 ? pa::launch_attend8_mma_f16_64(a, L.rows, L.hg, tmk, tmv, st) : pa::launch_attend8_mma_f16_128(a, L.rows, L.hg, tmk, tmv, st);
    return to_status(e);
}

int32_t run_umma(pa::Attend8Args &a, const pa_dims *d, void *stream) {
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    const bool bf16 = d->kv_dtype == PA_BF16;
    CUtensorMap tmq;
    cudaError_t e = pa::cached_query_map(a.q, bf16, a.D, a.Hq, a.T, a.Hq / a.Hkv, &tmq);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = pa::launch_attend8_plan(a, st);
    if (e == cudaSuccess) e = bf16 ? pa::launch_attend8_umma_bf16(a, tmq, st) : pa::launch_attend8_umma_f16(a, tmq, st);
    return to_status(e);
}

void fill_write8(pa::Write8Args &a, const pa_dims *d, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                 const int64_t *slots, int32_t T, const pa_cache8 *c) {
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slots;
    a.k_cache = static_cast<uint8_t *>(c->k);
    a.v_cache = static_cast<uint8_t *>(c->v);
    a.k_scales = c->k_scales;
    a.v_scales = c->v_scales;
    a.T = T;
    a.Hkv = d->num_kv_heads;
    a.D = d->head_dim;
    a.B = d->block_size;
    a.N = d->num_blocks;
    a.num_axes = 1;
    a.mscale = 1.f;
}

}  // namespace

extern "C" {

int32_t pa_rope_write_kv8(const pa_dims *dims, const pa_rope *rope, const pa_axes *axes, const void *q, int64_t q_stride,
                          const void *k, int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                          const int64_t *slot_mapping, int32_t num_tokens, void *q_out, int64_t q_out_stride,
                          const pa_cache8 *cache, void *stream) {
    int32_t rc = check_shape8(dims);
    if (rc == PA_OK) rc = pa::check_rope(dims, rope, axes);
    if (rc != PA_OK) return rc;
    if (num_tokens < 0 || num_tokens > kMaxTokens8) return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    rc = check_cache8(cache);
    if (rc == PA_OK)
        rc = pa::check_rope_tokens(dims, rope, q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, num_tokens,
                                   q_out, q_out_stride);
    if (rc != PA_OK) return rc;
    pa::Write8Args a{};
    fill_write8(a, dims, k, k_stride, v, v_stride, slot_mapping, num_tokens, cache);
    a.q = q;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.Hq = dims->num_q_heads;
    a.positions = positions;
    a.pair_axis = axes ? axes->pair_axis : nullptr;
    a.num_axes = axes ? axes->num_axes : 1;
    a.freqs = rope->freqs;
    a.R = rope->rotary_dim;
    a.interleaved = rope->interleaved;
    a.mscale = rope->mscale;
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    return to_status(pa::launch_write8(a, dims->kv_dtype == PA_BF16, static_cast<cudaStream_t>(stream)));
}

int32_t pa_write_kv8(const pa_dims *dims, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     const int64_t *slot_mapping, int32_t num_tokens, const pa_cache8 *cache, void *stream) {
    int32_t rc = check_shape8(dims);
    if (rc != PA_OK) return rc;
    if (num_tokens < 0 || num_tokens > kMaxTokens8) return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    rc = check_cache8(cache);
    if (rc != PA_OK) return rc;
    const int64_t row = (int64_t)dims->num_kv_heads * dims->head_dim;
    if (!k || !v || !slot_mapping || k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return PA_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8)) return PA_ERR_INVALID;
    pa::Write8Args a{};
    fill_write8(a, dims, k, k_stride, v, v_stride, slot_mapping, num_tokens, cache);
    a.err = pa::device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    return to_status(pa::launch_write8(a, dims->kv_dtype == PA_BF16, static_cast<cudaStream_t>(stream)));
}

int32_t pa_copy_blocks8(const pa_dims *dims, const pa_cache8 *cache, const int64_t *src_dst_pairs, int32_t num_pairs,
                        void *stream) {
    int32_t rc = check_shape8(dims);
    if (rc != PA_OK) return rc;
    if (num_pairs < 0) return PA_ERR_INVALID;
    if (num_pairs == 0) return PA_OK;
    rc = check_cache8(cache);
    if (rc != PA_OK) return rc;
    if (!src_dst_pairs || !aligned(src_dst_pairs, 8)) return PA_ERR_INVALID;
    unsigned int *err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    const int64_t block_bytes = (int64_t)dims->num_kv_heads * dims->block_size * dims->head_dim;
    return to_status(pa::launch_copy_blocks8(static_cast<uint8_t *>(cache->k), static_cast<uint8_t *>(cache->v), cache->k_scales,
                                             cache->v_scales, src_dst_pairs, num_pairs, dims->num_blocks, block_bytes,
                                             dims->num_kv_heads, err, static_cast<cudaStream_t>(stream)));
}

size_t pa_decode8_workspace_bytes(const pa_dims *dims) {
    if (check_attend8(dims) != PA_OK || dims->num_seqs == 0) return 0;
    return decode_layout8(dims, nullptr).total;   // (a window may save the joins; what is left then needs less)
}

int32_t pa_decode8(const pa_dims *dims, const pa_window *window, const void *q, const pa_cache8 *cache,
                   const int32_t *block_tables, const int32_t *context_lens, float scale, void *out, int32_t out_dtype,
                   void *workspace, size_t workspace_bytes, void *stream) {
    int32_t rc = check_attend8(dims);
    if (rc == PA_OK) rc = check_window(window);
    if (rc != PA_OK) return rc;
    if (out_dtype != PA_F32 && out_dtype != dims->kv_dtype) return PA_ERR_INVALID;
    if (dims->num_seqs == 0) return PA_OK;
    rc = check_cache8(cache);
    if (rc != PA_OK) return rc;
    if (!q || !block_tables || !context_lens || !out) return PA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4)) return PA_ERR_INVALID;
    const Layout8 L = decode_layout8(dims, window);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)) return PA_ERR_INVALID;
    pa::Attend8Args a{};
    fill8(a, dims, window, q, cache, block_tables, context_lens, scale, out, out_dtype, L, workspace);
    a.T = dims->num_seqs;
    a.max_query_len = 1;
    return run_mma(a, dims, L, stream);
}

size_t pa_chunk8_workspace_bytes(const pa_dims *dims, int32_t num_tokens, int32_t max_query_len) {
    if (check_chunk8(dims, num_tokens, max_query_len) != PA_OK) return 0;
    // (a window may save the line; what is left then needs less)
    return chunk_layout8(dims, max_query_len, nullptr).total;
}

int32_t pa_chunk8(const pa_dims *dims, const pa_window *window, const void *q, const pa_cache8 *cache,
                  const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start, int32_t num_tokens,
                  int32_t max_query_len, float scale, void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
                  void *stream) {
    int32_t rc = check_chunk8(dims, num_tokens, max_query_len);
    if (rc == PA_OK) rc = check_window(window);
    if (rc != PA_OK) return rc;
    if (out_dtype != PA_F32 && out_dtype != dims->kv_dtype) return PA_ERR_INVALID;
    if (dims->num_seqs == 0 || num_tokens == 0) return PA_OK;
    rc = check_cache8(cache);
    if (rc != PA_OK) return rc;
    if (!q || !block_tables || !context_lens || !query_start || !out) return PA_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4))
        return PA_ERR_INVALID;
    const Layout8 L = chunk_layout8(dims, max_query_len, window);
    if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256)) return PA_ERR_INVALID;
    pa::Attend8Args a{};
    fill8(a, dims, window, q, cache, block_tables, context_lens, scale, out, out_dtype, L, workspace);
    a.query_start = query_start;
    a.T = num_tokens;
    a.max_query_len = max_query_len;
    return L.tiles ? run_umma(a, dims, stream) : run_mma(a, dims, L, stream);
}

}  // extern "C"
