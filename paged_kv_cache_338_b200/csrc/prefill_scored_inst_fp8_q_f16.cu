// Instantiations of the modified-score chunk attention: f16 queries, E4M3 cache.
#include "prefill_scored.cuh"

cudaError_t ps::launch_fp8_q_f16(const Launch& a, int) {
    return launch_mod<PA_F16, true, 128>(a);
}
