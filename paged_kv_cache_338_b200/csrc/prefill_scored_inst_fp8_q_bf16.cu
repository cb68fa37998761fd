// Instantiations of the modified-score chunk attention: bf16 queries, E4M3 cache.
#include "prefill_scored.cuh"

cudaError_t ps::launch_fp8_q_bf16(const Launch& a, int) {
    return launch_mod<PA_BF16, true, 128>(a);
}
