// pa_attend8_mma_f16_64.cu -- decode and short chunks over the 8-bit cache, f16 queries, head_dim 64.
#include "pa_attend8_mma.cuh"

namespace pa {

cudaError_t launch_attend8_mma_f16_64(const Attend8Args &a, Rows8 rows, int hg, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    return dispatch_attend8<__half, 64>(a, rows, hg, tmk, tmv, st);
}

}  // namespace pa
