// pa_chunk_scored_umma_f16.cu -- scored chunk attention for f16 KV caches, the
// tcgen05 kernel (a translation unit of its own, to compile in parallel).
#include "pa_chunk_scored_umma.cuh"

namespace pa {
cudaError_t launch_scored_umma_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return dispatch_scored_umma<__half>(a, tmk, tmv, tmq, tmo, st);
}
}  // namespace pa
