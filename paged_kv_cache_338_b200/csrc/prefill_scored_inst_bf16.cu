// Instantiations of the modified-score chunk attention: bf16 queries and cache.
#include "prefill_scored.cuh"

cudaError_t ps::launch_bf16(const Launch& a, int D) {
    return D == 64 ? launch_mod<PA_BF16, false, 64>(a) : launch_mod<PA_BF16, false, 128>(a);
}
