// pa_attend8_mma_bf16.cu -- decode and short chunks over the 8-bit cache, bf16 queries.
#include "pa_attend8_mma.cuh"

namespace pa {

cudaError_t launch_attend8_mma_bf16(const Attend8Args &a, int team, const CUtensorMap &tmk, const CUtensorMap &tmv, cudaStream_t st) {
    const cudaError_t e = dispatch_attend8<__nv_bfloat16>(a, team, tmk, tmv, st);
    return e != cudaSuccess ? e : dispatch_merge8<__nv_bfloat16>(a, team, st);
}

}  // namespace pa
