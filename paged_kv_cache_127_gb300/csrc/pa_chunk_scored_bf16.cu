// pa_chunk_scored_bf16.cu -- scored chunk attention for bf16 KV caches, the
// mma.sync kernel (a translation unit of its own, to compile in parallel).
#include "pa_chunk_scored_mma.cuh"

namespace pa {
cudaError_t launch_scored_chunk_bf16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                     cudaStream_t st) {
    return dispatch_scored_chunk<__nv_bfloat16>(a, tmk, tmv, st);
}
}  // namespace pa
