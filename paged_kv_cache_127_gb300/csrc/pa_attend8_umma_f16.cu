// pa_attend8_umma_f16.cu -- long chunks over the 8-bit cache, f16 queries.
#include "pa_attend8_umma.cuh"

namespace pa {

cudaError_t launch_attend8_umma_f16(const Attend8Args &a, const CUtensorMap &tmq, cudaStream_t st) {
    return dispatch_umma8<__half>(a, tmq, st);
}

}  // namespace pa
