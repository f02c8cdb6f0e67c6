// pa_evict.cu -- eviction by summed attention weights: which tokens each KV head
// keeps, and their copy to fresh blocks.
//
// Selection, one CTA per (sequence, KV head): of the n = len - recent older
// tokens the m = keep - recent with the largest sums.  Sums become 32-bit keys
// whose unsigned order is theirs (NaN lowest, -0 as +0), and the m-th largest
// key is found by radix selection, a histogram of 8 bits per pass.  A token is
// kept if its key is larger, or equal and among the first `ties` equal ones, or
// if it is recent; a block-wide scan in index order gives each kept token its
// new position, written to the move list, and its sum to the new place.
// Copy: one thread per 16 bytes of a kept key or value row.
#include "pa_device.cuh"
#include "pa_scored.h"

namespace pa {

namespace {

constexpr int kSelThreads = 1024;

// Unsigned order of the keys = order of the sums; NaN below everything.
__device__ __forceinline__ uint32_t sum_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of v over the block (1024 threads); *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[wid] = incl;
    __syncthreads();
    if (wid == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const int base = wid > 0 ? warp_sums[wid - 1] : 0;
    *total = warp_sums[31];
    __syncthreads();
    return base + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int warp_sums[32];
    __shared__ uint32_t s_key;
    __shared__ int s_want;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x;
    const int cap = a.max_blocks * a.B;
    int len = a.lens[s], keep = a.keep_lens[s];
    if (len < 0 || len > cap || keep < 0) {
        if (tid == 0 && h == 0) set_error(a.err, PA_DEVERR_BAD_LEN);
        len = len < 0 ? 0 : (len > cap ? cap : len);
        if (keep < 0) keep = len;
    }
    const int row = a.sum_rows ? a.sum_rows[s] : s;
    const bool bad_row = row < 0 || row >= a.sum_num_rows;
    if (bad_row) {
        if (tid == 0 && h == 0) set_error(a.err, PA_DEVERR_BAD_ROW);
        keep = len;
    }
    const int now = min(len, keep);
    if (tid == 0) {
        a.counts[blockIdx.x] = len > keep ? keep : 0;
        if (h == 0) a.new_lens[s] = now;
    }
    if (bad_row) return;
    const float *in = a.sums + ((size_t)row * a.Hkv + h) * a.sum_cols;
    float *out = a.sums_out + ((size_t)row * a.Hkv + h) * a.sum_cols;
    if (len <= keep) {
        for (int j = tid; j < a.sum_cols; j += blockDim.x) out[j] = j < now ? in[j] : 0.f;
        return;
    }
    const int recent = min(a.recent, keep);
    const int n = len - recent, m = keep - recent;  // m < n
    // the m-th largest key, 8 bits at a time; `want` of the keys that share the prefix so far
    uint32_t prefix = 0;
    int want = m;
    if (m > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            const uint32_t high = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j = tid; j < n; j += blockDim.x) {
                const uint32_t k = sum_key(in[j]);
                if ((k & high) == prefix) atomicAdd(&hist[k >> shift & 255u], 1);
            }
            __syncthreads();
            // bins from the largest down: the one that holds the want-th key
            int total;
            const int v = tid < 256 ? hist[255 - tid] : 0;
            const int before = block_scan(v, warp_sums, &total);
            if (tid < 256 && before < want && want <= before + v) {
                s_key = prefix | (uint32_t)(255 - tid) << shift;
                s_want = want - before;
            }
            __syncthreads();
            prefix = s_key;
            want = s_want;
            __syncthreads();
        }
    }
    // kept tokens in index order; `want` of those equal to the m-th largest key
    int *list = a.list + ((size_t)s * a.Hkv + h) * cap;
    int kept = 0, equal = 0;
    for (int j0 = 0; j0 < len; j0 += kSelThreads) {
        const int j = j0 + tid;
        const float x = j < len ? in[j] : 0.f;
        const uint32_t k = sum_key(x);
        const bool old = j < n, eq = old && m > 0 && k == prefix;
        int total;
        const int eq_before = equal + block_scan(eq ? 1 : 0, warp_sums, &total);
        equal += total;
        const bool keep_it = (old && m > 0 && (k > prefix || (eq && eq_before < want))) || (j >= n && j < len);
        const int at = kept + block_scan(keep_it ? 1 : 0, warp_sums, &total);
        kept += total;
        // `at` <= j, and every sum of this tile has been read: in place is safe
        if (keep_it) {
            list[at] = j;
            out[at] = x;
        }
    }
    __syncthreads();
    for (int j = now + tid; j < a.sum_cols; j += blockDim.x) out[j] = 0.f;
}

// grid: (tiles of kMoveRows rows, sequence * Hkv, {K, V})
constexpr int kMoveRows = 64;
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a, int chunks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int sh = blockIdx.y, s = sh / a.Hkv, h = sh % a.Hkv;
    const int count = a.counts[sh];
    const int r0 = blockIdx.x * kMoveRows;
    if (r0 >= count) return;
    const int cap = a.max_blocks * a.B;
    uint4 *cache = static_cast<uint4 *>(blockIdx.z ? a.v_cache : a.k_cache);
    const int32_t *from = a.tables + (size_t)s * a.max_blocks;
    const int32_t *to = a.new_tables + (size_t)s * a.max_blocks;
    const int *list = a.list + (size_t)sh * cap;
    const int rows = min(kMoveRows, count - r0);
    for (int u = threadIdx.x; u < rows * chunks; u += blockDim.x) {
        const int r = r0 + u / chunks, c = u % chunks;
        const int j = list[r];
        const int fb = from[j / a.B], tb = to[r / a.B];
        if (fb < 0 || fb >= a.N || tb < 0 || tb >= a.N) {
            set_error(a.err, PA_DEVERR_BAD_BLOCK);
            continue;
        }
        cache[(((size_t)tb * a.Hkv + h) * a.B + r % a.B) * chunks + c] =
            cache[(((size_t)fb * a.Hkv + h) * a.B + j % a.B) * chunks + c];
    }
}

cudaError_t launch_pdl(void (*kernel)(EvictArgs), dim3 grid, int threads, const EvictArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t st) {
    if (a.S == 0) return cudaSuccess;
    cudaError_t e = launch_pdl(evict_select_kernel, dim3((unsigned)(a.S * a.Hkv)), kSelThreads, a, st);
    if (e != cudaSuccess) return e;
    const int cap = a.max_blocks * a.B;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cap + kMoveRows - 1) / kMoveRows), (unsigned)(a.S * a.Hkv), 2u);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, a, a.row_bytes / 16);
}

}  // namespace pa
