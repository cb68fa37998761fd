// Instantiations of the few-row chunk attention: f16 queries and cache.
#include "prefill_few.cuh"

cudaError_t ps::launch_few_f16(const Launch& a, int D) {
    return D == 64 ? launch_few<PA_F16, false, 64>(a) : launch_few<PA_F16, false, 128>(a);
}
