// Norm of every query and key head, rotation by position and cache append in
// one pass (pa_norm_rope_append).
//
// What is computed, per new token t at position p and per head row x of D
// elements (q and k; v is only written to the cache):
//     y = x * (1 / sqrt(mean(x^2) + eps)) * (w + weight_offset)   (w given)
//     (a, b) -> (a cos - b sin, b cos + a sin)   for the rot_dim / 2 pairs of
//               the row, cos and sin from row p of the caller's table
// all in fp32, rounded once: q rows to q_out, k and v rows to the token's
// cache slot (the same dtype, or E4M3 of x / scale as pa_reshape_and_cache).
//
// Layout.  A lane holds 16 elements of a row as two 8-element chunks, chosen
// so that both members of every rotated pair sit in the same lane (chunk c
// and chunk c + rot_dim / 16 of the rotated part; two neighbouring chunks
// past it).  D / 16 lanes hold a row, a warp 32 * 16 / D rows, and a row's sum
// of squares takes log2(D / 16) shuffles and the rotation none.  A warp works
// on one token, so a lane loads its 8 cosines and sines once for all heads.
// Every global access is 16 bytes a lane (8 for E4M3), kPasses passes of
// loads in flight before the first use.
//
// The work is one read of q, k, v and one write of each: HBM-bound for many
// tokens (32768 of 32/8 heads of 128, bf16: 149 us, 5.5 TB/s; into E4M3 152 us),
// latency-bound for a decode step (8 tokens: 3.1 us), where the passes of a token
// are spread over `split` warps.  Rows are worked on two elements an instruction:
// with one the issue slots were half taken and the registers held 12 warps an SM.
#include <cuda_runtime.h>

#include <cmath>

#include "pa_internal.h"
#include "tc_device.cuh"

namespace {

using namespace pa::dev;

constexpr int kThreads = 128;
// Passes whose loads are in flight, and CTAs an SM holds at least (which bounds the
// registers).  32768 tokens, 32/8 heads of 128, bf16: 2 passes and 4 CTAs 150 us, 2 and
// 5 166 (spills), 4 and 3 170, 1 and 6 186.
constexpr int kPasses = 2;
constexpr int kBlocks = 4;

struct Params {
    uint8_t* q_out;
    const uint8_t *q, *k, *v;
    long long q_out_stride, q_stride, k_stride, v_stride;   // bytes between tokens
    const uint8_t *q_weight, *k_weight;                      // [D], or NULL: no norm
    float eps, weight_offset;
    const float* cos_sin;                                    // [table_rows, rot_dim]
    long long table_rows;
    const int64_t* positions;
    int rot_dim, interleaved;
    uint8_t *kc, *vc;
    const int64_t* slots;
    long long nslots;
    float k_scale, v_scale, k_inverse, v_inverse;
    unsigned int* err;
    int T, Hq, Hkv;
    int split;                                               // warps per token
};

// 8 consecutive elements at element index e of a row, as raw 16-byte words.
template <int DT> struct Raw8;
template <> struct Raw8<PA_F32> {
    uint4 a, b;
    __device__ __forceinline__ void load(const uint8_t* row, int e) {
        a = *reinterpret_cast<const uint4*>(row + e * 4);
        b = *reinterpret_cast<const uint4*>(row + e * 4 + 16);
    }
    __device__ __forceinline__ void store(uint8_t* row, int e) const {
        *reinterpret_cast<uint4*>(row + e * 4) = a;
        *reinterpret_cast<uint4*>(row + e * 4 + 16) = b;
    }
    __device__ __forceinline__ void to_float(float* f) const {
        Chunk<PA_F32>::to_float(a, f);
        Chunk<PA_F32>::to_float(b, f + 4);
    }
    __device__ __forceinline__ void from_float(const float* f) {
        a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3]));
        b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                       __float_as_uint(f[7]));
    }
};
template <int DT> struct Raw16 {
    uint4 a;
    __device__ __forceinline__ void load(const uint8_t* row, int e) {
        a = *reinterpret_cast<const uint4*>(row + e * 2);
    }
    __device__ __forceinline__ void store(uint8_t* row, int e) const {
        *reinterpret_cast<uint4*>(row + e * 2) = a;
    }
    __device__ __forceinline__ void to_float(float* f) const { Chunk<DT>::to_float(a, f); }
    __device__ __forceinline__ static uint32_t pack(float x, float y) {
        if constexpr (DT == PA_BF16) {
            __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            return *reinterpret_cast<uint32_t*>(&h);
        } else {
            __half2 h = __floats2half2_rn(x, y);
            return *reinterpret_cast<uint32_t*>(&h);
        }
    }
    __device__ __forceinline__ void from_float(const float* f) {
        a = make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
    }
};
template <> struct Raw8<PA_F16> : Raw16<PA_F16> {};
template <> struct Raw8<PA_BF16> : Raw16<PA_BF16> {};

// x / scale in binary32, to nearest even, as the cache append divides.  With
// `inverse` = 1 / scale rounded to nearest (0: a scale outside 2^-60..2^60) one
// residual step gives the correctly rounded quotient (Markstein's theorem).  Past 512
// a quotient saturates whatever its last bits, and below 2^-12 it is a zero code of
// its sign (which the step would lose), so both ends go without.
__device__ __forceinline__ float quotient(float x, float scale, float inverse) {
    const float q = x * inverse;
    const float r = fmaf(fmaf(-q, scale, x), inverse, q);
    return fabsf(q) < 512.f && fabsf(q) > 0x1p-12f ? r : q;
}

// 8 floats to 8 E4M3 codes of x / scale, to nearest even, saturating.
__device__ __forceinline__ uint2 to_e4m3x8(const float* f, float scale, float inverse) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        w[k] = 0;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float a = f[4 * k + j], b = f[4 * k + j + 1];
            const float2 y = inverse != 0.f
                                 ? make_float2(quotient(a, scale, inverse), quotient(b, scale, inverse))
                                 : make_float2(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
            w[k] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (8 * j);
        }
    }
    return make_uint2(w[0], w[1]);
}

// The passes [lo, hi) of one kind of a token (KIND 0 queries, 1 keys, 2 values):
// kPasses batches of loads before the first use.  A pass is ROWS heads.
template <int IN, bool TO_FP8, int D, int KIND>
__device__ __forceinline__ void token_passes(const Params& p, const uint8_t* src, uint8_t* dst, int lo,
                                             int hi, int ea, int eb, bool turns, const float* cs,
                                             const float* sn, const float2* w, bool norm) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    constexpr int E = Storage<IN>::bytes;
    constexpr bool CODES = TO_FP8 && KIND > 0;     // E4M3 out
    constexpr int EO = CODES ? 1 : E;
    const int heads = KIND == 0 ? p.Hq : p.Hkv;
    const int row = (threadIdx.x & 31) / LANES;
#pragma unroll 1
    for (int pb = lo; pb < hi; pb += kPasses) {
        Raw8<IN> ra[kPasses], rb[kPasses];
#pragma unroll
        for (int u = 0; u < kPasses; ++u) {
            const int h = (pb + u) * ROWS + row;
            if (pb + u < hi && h < heads) {
                ra[u].load(src + (size_t)h * D * E, ea);
                rb[u].load(src + (size_t)h * D * E, eb);
            }
        }
#pragma unroll
        for (int u = 0; u < kPasses; ++u) {
            if (pb + u >= hi) break;               // warp-uniform
            const int h = (pb + u) * ROWS + row;
            uint8_t* out = dst + (size_t)h * D * EO;
            if constexpr (KIND == 2 && !TO_FP8) {  // a value row goes as it came
                if (h < heads) {
                    ra[u].store(out, ea);
                    rb[u].store(out, eb);
                }
            } else {
                float f[16];
                ra[u].to_float(f);
                rb[u].to_float(f + 8);
                if constexpr (KIND < 2) {
                    float2 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = make_float2(f[2 * i], f[2 * i + 1]);
                    if (norm) {                    // warp-uniform
                        float2 ss[2] = {};
#pragma unroll
                        for (int i = 0; i < 8; ++i) ss[i & 1] = fma2(y[i], y[i], ss[i & 1]);
                        float sum = (ss[0].x + ss[0].y) + (ss[1].x + ss[1].y);
#pragma unroll
                        for (int x = LANES / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                        const float inv = rsqrtf(fmaf(sum, 1.f / D, p.eps));
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = mul2(mul2(y[i], make_float2(inv, inv)), w[i]);
                    }
                    if (turns) {
                        if (p.interleaved) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float a = y[i].x, b = y[i].y;
                                y[i] = make_float2(a * cs[i] - b * sn[i], b * cs[i] + a * sn[i]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 c = make_float2(cs[2 * i], cs[2 * i + 1]);
                                const float2 s = make_float2(sn[2 * i], sn[2 * i + 1]);
                                const float2 a = y[i], b = y[4 + i];
                                y[i] = fma2(a, c, mul2(b, make_float2(-s.x, -s.y)));
                                y[4 + i] = fma2(b, c, mul2(a, s));
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[2 * i] = y[i].x, f[2 * i + 1] = y[i].y;
                }
                if (h >= heads) continue;
                if constexpr (CODES) {
                    const float sc = KIND == 1 ? p.k_scale : p.v_scale;
                    const float inv = KIND == 1 ? p.k_inverse : p.v_inverse;
                    *reinterpret_cast<uint2*>(out + ea) = to_e4m3x8(f, sc, inv);
                    *reinterpret_cast<uint2*>(out + eb) = to_e4m3x8(f + 8, sc, inv);
                } else {
                    ra[u].from_float(f);
                    rb[u].from_float(f + 8);
                    ra[u].store(out, ea);
                    rb[u].store(out, eb);
                }
            }
        }
    }
}

// One warp: its share of the passes of a token (the query heads' first, then the
// key heads', then the value heads'), then of the token `stride` units on.
template <int IN, bool TO_FP8, int D>
__global__ void __launch_bounds__(kThreads, IN == PA_F32 ? 3 : kBlocks) norm_rope_append_kernel(const Params p) {
    constexpr int LANES = D / 16;                 // lanes of a row
    constexpr int ROWS = 32 / LANES;              // rows of a pass
    constexpr int EC = TO_FP8 ? 1 : Storage<IN>::bytes;
    grid_dependency_wait();        // launched as a dependent of the kernel before it
    launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane % LANES;
    const long long units = (long long)p.T * p.split;
    const long long stride = (long long)gridDim.x * (kThreads / 32);
    const int nq = (p.Hq + ROWS - 1) / ROWS, nkv = (p.Hkv + ROWS - 1) / ROWS;
    const int passes = nq + 2 * nkv;

    // this lane's two chunks of a row, in elements
    const int half = p.rot_dim / 16;              // lanes that rotate
    const bool turns = sub < half;
    const int ea = turns ? 8 * sub : p.rot_dim + 16 * (sub - half);
    const int eb = turns ? p.rot_dim / 2 + 8 * sub : ea + 8;
    // first cosine of the lane's pairs 0-3 and 4-7: pairs (e, e + rot/2) have index
    // e, adjacent pairs (2j, 2j + 1) index j
    const int j0 = p.interleaved ? ea / 2 : ea, j1 = p.interleaved ? eb / 2 : ea + 4;

    for (long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); unit < units;
         unit += stride) {
        const long long t = unit / p.split;
        const int part = (int)(unit % p.split);
        const int p0 = (int)((long long)passes * part / p.split);
        const int p1 = (int)((long long)passes * (part + 1) / p.split);
        const int64_t slot = p.slots[t];
        const int64_t pos = half > 0 ? p.positions[t] : 0;
        const bool write = slot >= 0 && slot < p.nslots;
        if (slot >= p.nslots && lane == 0) raise_error(p.err, PA_DEV_BAD_SLOT);
        if (half > 0 && (pos < 0 || pos >= p.table_rows)) {   // warp-uniform: the token is skipped
            if (lane == 0) raise_error(p.err, PA_DEV_BAD_POSITION);
            continue;
        }
        float4 c0 = {}, c1 = {}, s0 = {}, s1 = {};
        if (turns) {
            const float* tr = p.cos_sin + pos * p.rot_dim;
            c0 = *reinterpret_cast<const float4*>(tr + j0);
            c1 = *reinterpret_cast<const float4*>(tr + j1);
            s0 = *reinterpret_cast<const float4*>(tr + p.rot_dim / 2 + j0);
            s1 = *reinterpret_cast<const float4*>(tr + p.rot_dim / 2 + j1);
        }
        const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        float2 w[8];
        auto weights = [&](const uint8_t* src) {
            if (!src) return false;
            Raw8<IN> a, b;
            float f[16];
            a.load(src, ea);
            b.load(src, eb);
            a.to_float(f);
            b.to_float(f + 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = make_float2(f[2 * i] + p.weight_offset, f[2 * i + 1] + p.weight_offset);
            return true;
        };
        const size_t cache = write ? (size_t)slot * p.Hkv * D * EC : 0;
        if (p0 < nq) {
            const bool norm = weights(p.q_weight);
            token_passes<IN, TO_FP8, D, 0>(p, p.q + t * p.q_stride, p.q_out + t * p.q_out_stride, p0,
                                           min(p1, nq), ea, eb, turns, cs, sn, w, norm);
        }
        if (write && p1 > nq && p0 < nq + nkv) {
            const bool norm = weights(p.k_weight);
            token_passes<IN, TO_FP8, D, 1>(p, p.k + t * p.k_stride, p.kc + cache, max(p0 - nq, 0),
                                           min(p1 - nq, nkv), ea, eb, turns, cs, sn, w, norm);
        }
        if (write && p1 > nq + nkv)
            token_passes<IN, TO_FP8, D, 2>(p, p.v + t * p.v_stride, p.vc + cache, max(p0 - nq - nkv, 0),
                                           p1 - nq - nkv, ea, eb, turns, cs, sn, w, false);
    }
}

template <int IN, bool TO_FP8, int D>
cudaError_t launch(Params p, cudaStream_t st) {
    constexpr int ROWS = 32 * 16 / D;
    constexpr long long per = kThreads / 32;
    const int passes = (p.Hq + ROWS - 1) / ROWS + 2 * ((p.Hkv + ROWS - 1) / ROWS);
    // Enough warps to fill the GPU (16 per SM) where the tokens alone do not: down
    // to one pass a warp.  Where there are more than the GPU holds at once, a warp
    // takes several tokens (32768 tokens: 149 us, with four times the CTAs 150, with
    // sixteen times 156).
    const long long want = 148LL * 16;
    long long split = (want + p.T - 1) / p.T;
    p.split = (int)(split < passes ? split : passes);
    const long long blocks = ((long long)p.T * p.split + per - 1) / per;
    int resident = 0;
    const cudaError_t e = occupancy<norm_rope_append_kernel<IN, TO_FP8, D>>(&resident, kThreads, 0);
    if (e != cudaSuccess) return e;
    const long long most = 148LL * (resident > 0 ? resident : 1);
    return launch_pdl(norm_rope_append_kernel<IN, TO_FP8, D>, dim3((unsigned)(blocks < most ? blocks : most)),
                      dim3(kThreads), 0, st, p);
}

template <int IN, bool TO_FP8>
cudaError_t launch_dim(const Params& p, int D, cudaStream_t st) {
    switch (D) {
    case 64: return launch<IN, TO_FP8, 64>(p, st);
    case 128: return launch<IN, TO_FP8, 128>(p, st);
    case 256: return launch<IN, TO_FP8, 256>(p, st);
    }
    return cudaErrorNotSupported;
}

// 1 / scale to nearest, 0 where a quotient by it may leave the normal range.
float inverse_of(float scale) {
    return scale >= 0x1p-60f && scale <= 0x1p60f ? 1.f / scale : 0.f;
}

}  // namespace

using pa::fail;

extern "C" pa_status pa_norm_rope_append(
    void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
    int64_t k_stride, const void* v, int64_t v_stride, pa_dtype in_dt, const void* q_weight,
    const void* k_weight, float eps, float weight_offset, const float* cos_sin,
    int64_t table_rows, const int64_t* positions, int rot_dim, int interleaved, void* key_cache,
    void* value_cache, pa_dtype cache_dt, const int64_t* slot_mapping, int T, int Hq, int Hkv,
    int D, int bs, int64_t NB, float k_scale, float v_scale, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_norm_rope_append");
    pa::clear_error();
    if (!pa::valid_dtype(in_dt) || !pa::valid_dtype(cache_dt))
        return fail(PA_ERR_INVALID_ARG, "bad dtype");
    if (in_dt == PA_FP8_E4M3 || !(cache_dt == in_dt || cache_dt == PA_FP8_E4M3))
        return fail(PA_ERR_UNSUPPORTED, "norm and rotation from dtype %d into dtype %d", in_dt,
                    cache_dt);
    if (T < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || bs <= 0 || NB <= 0)
        return fail(PA_ERR_INVALID_ARG, "negative or zero size");
    if (D != 64 && D != 128 && D != 256)
        return fail(PA_ERR_UNSUPPORTED, "head size %d (64, 128 or 256)", D);
    if (NB > (1LL << 62) / bs) return fail(PA_ERR_INVALID_ARG, "NB * bs overflows");
    if (rot_dim < 0 || rot_dim > D) return fail(PA_ERR_INVALID_ARG, "rot_dim %d outside [0, D]", rot_dim);
    if (rot_dim % 16)
        return fail(PA_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 16", rot_dim);
    if (!(std::isfinite(eps) && eps >= 0.f) || !std::isfinite(weight_offset))
        return fail(PA_ERR_INVALID_ARG, "eps must be finite and >= 0, weight_offset finite");
    if (!(std::isfinite(k_scale) && k_scale > 0 && std::isfinite(v_scale) && v_scale > 0))
        return fail(PA_ERR_INVALID_ARG, "scales must be finite and > 0");
    if (cache_dt != PA_FP8_E4M3 && (k_scale != 1.f || v_scale != 1.f))
        return fail(PA_ERR_INVALID_ARG, "k_scale / v_scale apply to fp8 caches only");
    const int e = pa::elem_size(in_dt);
    const int64_t strides[4] = {q_out_stride, q_stride, k_stride, v_stride};
    for (int i = 0; i < 4; ++i) {
        const int64_t row = (int64_t)(i < 2 ? Hq : Hkv) * D;
        if (strides[i] < row || strides[i] > (1LL << 40))
            return fail(PA_ERR_INVALID_ARG, "a token stride of %lld elements holds no row of %lld",
                        (long long)strides[i], (long long)row);
        if (strides[i] * e % 16)
            return fail(PA_ERR_INVALID_ARG, "token strides must be multiples of 16 bytes");
    }
    if (T == 0) return PA_OK;
    if (!q_out || !q || !k || !v || !key_cache || !value_cache || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (rot_dim > 0 && (!cos_sin || !positions || table_rows <= 0))
        return fail(PA_ERR_INVALID_ARG, "a rotation needs cos_sin, table_rows > 0 and positions");
    if (!pa::aligned16(q_out) || !pa::aligned16(q) || !pa::aligned16(k) || !pa::aligned16(v) ||
        !pa::aligned16(key_cache) || !pa::aligned16(value_cache) ||
        (q_weight && !pa::aligned16(q_weight)) || (k_weight && !pa::aligned16(k_weight)) ||
        (rot_dim > 0 && !pa::aligned16(cos_sin)))
        return fail(PA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;

    Params p = {};
    p.q_out = static_cast<uint8_t*>(q_out);
    p.q = static_cast<const uint8_t*>(q);
    p.k = static_cast<const uint8_t*>(k);
    p.v = static_cast<const uint8_t*>(v);
    p.q_out_stride = q_out_stride * e;
    p.q_stride = q_stride * e;
    p.k_stride = k_stride * e;
    p.v_stride = v_stride * e;
    p.q_weight = static_cast<const uint8_t*>(q_weight);
    p.k_weight = static_cast<const uint8_t*>(k_weight);
    p.eps = eps;
    p.weight_offset = weight_offset;
    p.cos_sin = cos_sin;
    p.table_rows = table_rows;
    p.positions = positions;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved ? 1 : 0;
    p.kc = static_cast<uint8_t*>(key_cache);
    p.vc = static_cast<uint8_t*>(value_cache);
    p.slots = slot_mapping;
    p.nslots = NB * bs;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_inverse = inverse_of(k_scale);
    p.v_inverse = inverse_of(v_scale);
    p.err = err;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool fp8 = cache_dt == PA_FP8_E4M3;
    cudaError_t ce;
    switch (in_dt) {
    case PA_F32: ce = fp8 ? launch_dim<PA_F32, true>(p, D, st) : launch_dim<PA_F32, false>(p, D, st); break;
    case PA_F16: ce = fp8 ? launch_dim<PA_F16, true>(p, D, st) : launch_dim<PA_F16, false>(p, D, st); break;
    default: ce = fp8 ? launch_dim<PA_BF16, true>(p, D, st) : launch_dim<PA_BF16, false>(p, D, st); break;
    }
    if (ce != cudaSuccess) return pa::cuda_fail(ce, "norm and rotation launch");
    return PA_OK;
}
