// Instantiations of the few-row chunk attention: bf16 queries, E4M3 cache.
#include "prefill_few.cuh"

cudaError_t ps::launch_few_fp8_q_bf16(const Launch& a, int) {
    return launch_few<PA_BF16, true, 128>(a);
}
