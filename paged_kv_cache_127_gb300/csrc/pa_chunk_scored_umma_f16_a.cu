// pa_chunk_scored_umma_f16_a.cu -- scored chunk attention for f16 KV caches, the
// tcgen05 kernel: mask only, cap max (translation units of their own,
// to compile in parallel).
#include "pa_chunk_scored_umma.cuh"

namespace pa {
cudaError_t launch_scored_umma_f16_mask_only(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__half, kMaskOnly>(a, tmk, tmv, tmq, tmo, st);
}
cudaError_t launch_scored_umma_f16_cap_max(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__half, kCapMax>(a, tmk, tmv, tmq, tmo, st);
}
}  // namespace pa
