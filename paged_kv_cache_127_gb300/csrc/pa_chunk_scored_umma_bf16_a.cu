// pa_chunk_scored_umma_bf16_a.cu -- scored chunk attention for bf16 KV caches, the
// tcgen05 kernel: mask only, cap fixed (translation units of their own,
// to compile in parallel).
#include "pa_chunk_scored_umma.cuh"

namespace pa {
cudaError_t launch_scored_umma_bf16_mask_only(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__nv_bfloat16, kMaskOnly>(a, tmk, tmv, tmq, tmo, st);
}
cudaError_t launch_scored_umma_bf16_cap_fixed(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__nv_bfloat16, kCapFixed>(a, tmk, tmv, tmq, tmo, st);
}
}  // namespace pa
