// Instantiations of the few-row chunk attention: f16 queries, E4M3 cache.
#include "prefill_few.cuh"

cudaError_t ps::launch_few_fp8_q_f16(const Launch& a, int) {
    return launch_few<PA_F16, true, 128>(a);
}
