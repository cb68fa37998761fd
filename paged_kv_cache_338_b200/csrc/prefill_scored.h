// Between the host entry of pa_prefill_scored and its kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ps {

constexpr int kPairGroup = 16;    // adjacent tile pairs scheduled side by side

// Halves of a CTA of the kernel for many rows that wait for every phase of an operand
// slot, and so take part in freeing it.  With two query tiles both halves read every
// tile.  With one the halves take the even and the odd key tiles, K_j in slot 2j and V_j
// in slot 2j + 1 of the ring: a number of slots that 4 divides gives each half slots of
// its own, any other makes them share, and a half that let a slot be filled again before
// it had looked would wait for a phase that its own tile has to bring about.
constexpr int slot_halves(int slots, bool two_tiles) { return two_tiles || slots % 4 ? 2 : 1; }

struct Params {
    void* out;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start;
    const int32_t* key_start;     // [T] first visible key per new token, or NULL
    const int32_t* prefix_lens;   // [S] leading keys every new token sees, or NULL
    const float* slopes;          // [Hq], or NULL
    unsigned int* err;
    long long NB;
    int T, Hq, G, log2G, TQ, MB, bs, log2bs, max_qlen, max_ctx, n_pairs, pair_group;
    int window;                   // > 0: keys at distance >= window are not visible
    int part_tiles, max_parts;    // key tiles per part; parts of a row at most
    float sl;                     // scale * k_scale * log2 e, with a cap 4 * scale * k_scale / softcap
    float cap_log2;               // softcap * log2 e, 0: none
    float v_scale;
    float2* ws_ml;                // [T, Hq, max_parts] (m, l)
    float* ws_o;                  // [T, Hq, max_parts, D]
};

struct Launch {
    const CUtensorMap *mq, *mk, *mv;
    const Params* p;
    dim3 grid;
    int few;                      // columns of the few-row kernel (16 or 32), 0: the other one
    cudaStream_t stream;
};

cudaError_t launch_bf16(const Launch& a, int D);
cudaError_t launch_f16(const Launch& a, int D);
cudaError_t launch_fp8_q_bf16(const Launch& a, int D);
cudaError_t launch_fp8_q_f16(const Launch& a, int D);
cudaError_t launch_few_bf16(const Launch& a, int D);
cudaError_t launch_few_f16(const Launch& a, int D);
cudaError_t launch_few_fp8_q_bf16(const Launch& a, int D);
cudaError_t launch_few_fp8_q_f16(const Launch& a, int D);

}  // namespace ps
