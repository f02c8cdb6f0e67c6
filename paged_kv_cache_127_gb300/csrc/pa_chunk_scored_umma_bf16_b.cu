// pa_chunk_scored_umma_bf16_b.cu -- scored chunk attention for bf16 KV caches, the
// tcgen05 kernel: cap max, bias, general (translation units of their own,
// to compile in parallel).
#include "pa_chunk_scored_umma.cuh"

namespace pa {
cudaError_t launch_scored_umma_bf16_cap_max(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__nv_bfloat16, kCapMax>(a, tmk, tmv, tmq, tmo, st);
}
cudaError_t launch_scored_umma_bf16_bias(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__nv_bfloat16, kBias>(a, tmk, tmv, tmq, tmo, st);
}
cudaError_t launch_scored_umma_bf16_general(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    return launch_scored_umma<__nv_bfloat16, kGeneral>(a, tmk, tmv, tmq, tmo, st);
}
}  // namespace pa
