// pa_decode_scored_f16.cu -- scored tensor-core decode for f16 KV caches (a
// translation unit of its own so the dtypes compile in parallel).
#include "pa_decode_scored.cuh"

namespace pa {
cudaError_t launch_scored_decode_f16(const ScoredArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                                      cudaStream_t st) {
    return dispatch_scored_decode<__half>(a, tmk, tmv, st);
}
cudaError_t scored_decode_ctas_f16(const ScoredArgs &a, int *ctas) { return dispatch_scored_decode_ctas<__half>(a, ctas); }
}  // namespace pa
