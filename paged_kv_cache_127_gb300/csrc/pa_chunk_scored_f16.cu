// pa_chunk_scored_f16.cu -- scored chunk attention for f16 KV caches, the
// mma.sync kernel (a translation unit of its own, to compile in parallel).
#include "pa_chunk_scored_mma.cuh"

namespace pa {
cudaError_t launch_scored_chunk_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                     cudaStream_t st) {
    return dispatch_scored_chunk<__half>(a, tmk, tmv, st);
}
}  // namespace pa
