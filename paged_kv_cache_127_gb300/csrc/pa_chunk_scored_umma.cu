// pa_chunk_scored_umma.cu -- which of the tcgen05 kernels a scored chunk takes.
#include "pa_chunk_scored_umma.cuh"

namespace pa {

#define PA_SCORED_UMMA(name) \
    cudaError_t launch_scored_umma_##name(const ScoredArgs &, const CUtensorMap &, const CUtensorMap &, \
                                          const CUtensorMap &, const CUtensorMap &, cudaStream_t)
PA_SCORED_UMMA(bf16_mask_only);
PA_SCORED_UMMA(bf16_cap_fixed);
PA_SCORED_UMMA(bf16_cap_max);
PA_SCORED_UMMA(bf16_bias);
PA_SCORED_UMMA(bf16_general);
PA_SCORED_UMMA(f16_mask_only);
PA_SCORED_UMMA(f16_cap_max);
PA_SCORED_UMMA(f16_bias);
PA_SCORED_UMMA(f16_general);
#undef PA_SCORED_UMMA

cudaError_t launch_scored_umma_bf16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                    const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    switch (scored_mode(a, true)) {
        case kMaskOnly: return launch_scored_umma_bf16_mask_only(a, tmk, tmv, tmq, tmo, st);
        case kCapFixed: return launch_scored_umma_bf16_cap_fixed(a, tmk, tmv, tmq, tmo, st);
        case kCapMax: return launch_scored_umma_bf16_cap_max(a, tmk, tmv, tmq, tmo, st);
        case kBias: return launch_scored_umma_bf16_bias(a, tmk, tmv, tmq, tmo, st);
        default: return launch_scored_umma_bf16_general(a, tmk, tmv, tmq, tmo, st);
    }
}

cudaError_t launch_scored_umma_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                   const CUtensorMap &tmq, const CUtensorMap &tmo, cudaStream_t st) {
    switch (scored_mode(a, false)) {
        case kMaskOnly: return launch_scored_umma_f16_mask_only(a, tmk, tmv, tmq, tmo, st);
        case kCapMax: return launch_scored_umma_f16_cap_max(a, tmk, tmv, tmq, tmo, st);
        case kBias: return launch_scored_umma_f16_bias(a, tmk, tmv, tmq, tmo, st);
        default: return launch_scored_umma_f16_general(a, tmk, tmv, tmq, tmo, st);
    }
}

}  // namespace pa
