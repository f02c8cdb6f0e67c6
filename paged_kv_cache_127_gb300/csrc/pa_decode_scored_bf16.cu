// pa_decode_scored_bf16.cu -- scored tensor-core decode for bf16 KV caches (a
// translation unit of its own so the dtypes compile in parallel).
#include "pa_decode_scored.cuh"

namespace pa {
cudaError_t launch_scored_decode_bf16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                      cudaStream_t st) {
    return dispatch_scored_decode<__nv_bfloat16>(a, tmk, tmv, st);
}
cudaError_t scored_decode_ctas_bf16(const ScoredArgs &a, int *ctas) { return dispatch_scored_decode_ctas<__nv_bfloat16>(a, ctas); }
}  // namespace pa
