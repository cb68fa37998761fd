// Attention of a chunk of new tokens over the paged cache with modified scores
// and masks (pa_prefill_scored) on the 5th-generation tensor cores.
//
// What is computed, for new token t at position p of its sequence and key i:
//     x = <q, k_i>
//     z = softcap * tanh(scale * x / softcap)  (cap)   or   scale * x
//     z -= slope[h] * |i - p|                  (distance bias)
//     out = sum_i softmax(z)_i v_i over the keys lo <= i <= hi, with
//         lo = max(p - window + 1, key_start[t], 0), hi = max(p, prefix - 1, cut to n - 1)
// Every row sees one range of keys, so a tile needs a mask only where a range
// begins or ends in it, and tiles before every range or past it are not read.
//
// Tiling.  A query tile is 128 rows: TQ = 128 / G new tokens x the G query heads
// of one kv head.  A CTA serves two adjacent query tiles A and B (256 rows per
// K / V tile read), or, where B has no rows (a few proposed tokens on a long
// context), one: then A's warps take the even key tiles and B's warps the odd
// ones of the same rows, and A merges both states at the end, so the softmax of
// one key tile runs beside the products of the other.  Keys run in tiles of 128
// from the block of the first visible key on.  Per key tile j and half X:
//     S_X = Q K_j^T    tcgen05.mma, 128 x 128 x D, operands in shared memory
//     P_X = exp2(z - m)  one row per thread, rounded to the operand type and
//                        written over S_X in tensor memory
//     O_X += P_X V_j   tcgen05.mma, P from tensor memory
// m is raised (and O_X rescaled) only when a tile's maximum exceeds it by 8 in
// log2 units; between raises the probabilities stay below 2^8, the same softmax.
// With few CTAs the keys are split over CTAs too (`part_tiles` key tiles each):
// each writes its state (m, l, O) in fp32 and a second kernel joins them.
//
// 8-bit cache.  The copies bring E4M3 codes; four more warps widen them to f16
// (exactly) into the operand slots.  A bf16 query row is brought to f16 by a
// power of two of its own, which sets its largest element to 2^14..2^15 (an
// element 2^-29 of that and smaller loses bits, below fp32's own rounding of
// the sum), and its inverse multiplies the row's scores.
//
// Rounding.  Scores, maxima, sums and O are fp32.  Probabilities are rounded to the operand
// type, half a step (2^-9 of bf16, 2^-12 of f16) each: the MMA takes both operands in one
// type, V is stored in it, and together the errors come to about what the output's own
// rounding adds.  The row's sum takes them unrounded, off the way to P.V.
//
// Not-a-numbers.  A probability of zero times a non-finite value is no zero, so
// where a row does not see a key, that key's value must not meet the row in the
// product.  In tiles that some row masks, a warp looks through V (one multiply
// by zero per two elements) and sets non-finite elements to zero before the
// product; the epilogue then adds them back to the rows that do see their key,
// reading them from the cache.  Tiles that all rows see whole need neither.  The
// MMA warps do the look while they wait for P anyway (880 of its 2600 cycles).
//
// Warps: 0-3 and 4-7 softmax and epilogue of halves A and B; 8 copies; 9 and 10
// the MMAs of A and B, and the look through V; 11 completes their warpgroup; 8-bit:
// 12-15 widening.  The softmax warps w and w + 4 share a scheduler and take turns
// with their exponentials (A, B, A, ...), as in pa_prefill.  Tensor memory: S_A 0..127, O_A 128..255, S_B 256..383, O_B 384..511.  Every wait is
// bounded (2 s): then PA_DEV_WAIT_TIMEOUT is set and the CTA drains its copies
// and MMAs, frees its tensor memory and exits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "pa_internal.h"
#include "prefill_scored.h"
#include "tc_device.cuh"

namespace ps {

using namespace pa::dev;

constexpr int kBN = 128;          // keys per tile
constexpr int kSeg = 16384;       // 128 rows x 128 bytes: one operand segment
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;

template <bool FP8, int D>
struct Plan {
    static constexpr int NSEG = D / 64;              // 128-byte segments of an operand row
    static constexpr int TILE = NSEG * kSeg;         // 128 rows of D operand elements
    // operand slots, K_j and V_j in turn
    static constexpr int NS = FP8 ? 3 : D == 64 ? 8 : 4;
    static constexpr int RS = FP8 ? 4 : 0;           // slots of E4M3 codes
    static constexpr int Q = 0;
    static constexpr int OP = 2 * TILE;
    static constexpr int RAW = OP + NS * TILE;
    // fp8: row factors, 256 of both halves, or (without B) 128; and without B
    // 128 x (m, l) of half B behind those
    static constexpr int ROWSCALE = RAW + RS * kSeg;
    static constexpr int ML = ROWSCALE + 512;
    static constexpr int BAR = ML + 1024;
    // q_full, q_ready, full[NS], free[NS], raw_full[RS], raw_free[RS], per half
    // s_full, p_full, pv_done, o_full; drain, b_done; per half and softmax warp
    // the turn of its exponentials
    static constexpr int NBAR = 2 + 2 * NS + 2 * RS + 8 + 2 + 8;
    // tensor memory address, abort flag, dirty range, ranges of 8 warps, Stash
    static constexpr int MISC = BAR + NBAR * 8;
    static constexpr int BYTES = MISC + 192 + 1024;  // + alignment
    static_assert(BYTES <= 232448, "shared memory of one CTA");
    static constexpr int THREADS = FP8 ? 512 : 384;
    // setmaxnreg: softmax warps / the others.  The shares must fit what the
    // block was launched with (checked before the first launch).
    static constexpr int RSOFT = FP8 ? 200 : 208, ROTHER = FP8 ? 48 : 64;
    static constexpr int RTOTAL = 256 * RSOFT + (THREADS - 256) * ROTHER;
};

// The rows of one half of a CTA, as ranges over their visible keys.
struct Ranges {
    int minlo, maxlo, minhi, maxhi;
};
constexpr int kNoLo = INT_MAX, kNoHi = -1;

// The six-term fit beside kTanh4, |u| <= 4 (7e-7 in fp32 arithmetic); a probability is
// rounded to 2^-9 or 2^-12 afterwards.  Both are smooth in u, so scores near one
// another, the only ones that share a row's weight, are off by the same amount.
__device__ constexpr float kTanh6[6] = {0.24999985f, -0.0052076629f, 0.00012970150f,
                                        -3.1497602e-06f, 6.3869905e-08f, -7.3124384e-10f};

// What the epilogue needs of the setup, kept in shared memory meanwhile (the
// softmax loop needs the registers).
struct Stash {
    int q0, iA, g, part, parts, nt, kb, maxlo, minhi;
};

// 1 / x on the special-function unit (1 / infinity = 0).
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// min(a, b, c) in one instruction.
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// min(a, b), NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Whether any of 8 16-bit elements is infinite or NaN: zero times it is not zero.
template <int OT> __device__ __forceinline__ bool nonfinite(const uint4& w) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t acc = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (OT == PA_BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(v[i]), "r"(0u));
        else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(v[i]), "r"(0u));
    }
    return (acc & 0x7fff7fffu) != 0u;
}

// The same 8 elements with 0 in place of those.
template <int OT> __device__ __forceinline__ uint4 finite_only(const uint4& w) {
    constexpr uint32_t E = OT == PA_BF16 ? 0x7f80u : 0x7c00u;
    auto fix = [](uint32_t v) {
        return ((v & E) == E ? 0u : v & 0xffffu) | ((v >> 16 & E) == E ? 0u : v & 0xffff0000u);
    };
    return make_uint4(fix(w.x), fix(w.y), fix(w.z), fix(w.w));
}

// Four E4M3 codes to four halves (exact).
__device__ __forceinline__ uint2 widen(uint32_t codes) {
    uint2 h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
        : "=r"(h.x), "=r"(h.y)
        : "r"(codes));
    return h;
}

// Row r of a swizzled bf16 query tile to f16, in place, times a power of two
// that sets its largest finite element to 2^14..2^15 (infinities and NaN stay what
// they are); returns the inverse.
template <int D, int SEG = kSeg> __device__ __forceinline__ float row_to_f16(uint32_t tile, int r) {
    float top = 0.f;
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {
        float f[8];
        Chunk<PA_BF16>::to_float(lds128(tile + (i >> 3) * SEG + swz128(r, i & 7)), f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (fabsf(f[k]) <= 3.4e38f) top = fmaxf(top, fabsf(f[k]));
    }
    int sh = 0;                        // rows of zeros: as they are
    if (top > 0.f) sh = min(126, 14 - ((int)(__float_as_uint(top) >> 23) - 127));
    const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {
        const uint32_t at = tile + (i >> 3) * SEG + swz128(r, i & 7);
        float f[8];
        Chunk<PA_BF16>::to_float(lds128(at), f);
        sts128(at, make_uint4(pack2<PA_F16>(f[0] * up, f[1] * up), pack2<PA_F16>(f[2] * up, f[3] * up),
                              pack2<PA_F16>(f[4] * up, f[5] * up), pack2<PA_F16>(f[6] * up, f[7] * up)));
    }
    return __uint_as_float((uint32_t)(127 - sh) << 23);
}

// One element of a cache as float (E4M3 without its scale).
template <int DT> __device__ __forceinline__ float cache_value(const void* p, size_t i) {
    if constexpr (DT == PA_FP8_E4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[i], __NV_E4M3);
        return __half2float(__half(h));
    } else {
        return load_q<DT>(p, i);
    }
}

// tanh(u / 4) on the special-function unit: 1 - 2 / (1 + e^(u / 2)); past 2^30
// that is 1 in fp32.
__device__ __forceinline__ float tanh_quarter(float u) {
    return fmaf(-2.f, rcp(1.f + ex2(min_nan(u * (0.5f * kLog2e), 30.f))), 1.f);
}

// A pair of capped scores, cap * tanh(u / 4), right to within 7e-7 of each: kTanh6 up to
// |u| = 4, the special-function unit beyond (FAR: not all of the warp's are within 4.  What
// a score becomes does not depend on it, so neither on the scores beside it).
template <bool FAR> __device__ __forceinline__ float2 capped2(float2 u, float cap) {
    const float2 v = mul2(u, u);
    float2 y = make_float2(kTanh6[5], kTanh6[5]);
#pragma unroll
    for (int t = 4; t >= 0; --t) y = fma2(y, v, make_float2(kTanh6[t], kTanh6[t]));
    y = mul2(mul2(u, make_float2(cap, cap)), y);
    if constexpr (FAR) {
        if (!(fabsf(u.x) <= 4.f)) y.x = cap * tanh_quarter(u.x);
        if (!(fabsf(u.y) <= 4.f)) y.y = cap * tanh_quarter(u.y);
    }
    return y;
}

// cap * tanh(u / 4) by the fit of `terms` terms, as the exponentials' loops take it.
__device__ __forceinline__ float fitted(float u, float cap, int terms) {
    const float v = u * u;
    float y;
    if (terms == 4) {
        y = kTanh4[3] * cap;
#pragma unroll
        for (int t = 2; t >= 0; --t) y = fmaf(y, v, kTanh4[t] * cap);
    } else {
        y = kTanh6[5] * cap;
#pragma unroll
        for (int t = 4; t >= 0; --t) y = fmaf(y, v, kTanh6[t] * cap);
    }
    return u * y;
}

// The largest and the smallest of 32 values, as independent chains (NaN is passed over).
__device__ __forceinline__ float max32(const float* s) {
    float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < 32; k += 2) m[(k >> 1) & 3] = max3(m[(k >> 1) & 3], s[k], s[k + 1]);
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}
__device__ __forceinline__ float min32(const float* s) {
    float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < 32; k += 2) m[(k >> 1) & 3] = min3(m[(k >> 1) & 3], s[k], s[k + 1]);
    return fminf(min3(m[0], m[1], m[2]), m[3]);
}

// Bits a..b (inclusive, any integers) of 32-bit word g.
__device__ __forceinline__ uint32_t range_word(int a, int b, int g) {
    a -= 32 * g;
    b -= 32 * g;
    if (b < 0 || a > 31 || a > b) return 0u;
    const uint32_t up = b >= 31 ? ~0u : (2u << b) - 1u;
    return a <= 0 ? up : up & (~0u << a);
}

// 32 outputs o * f from element `at` on.
template <int QT> __device__ __forceinline__ void store32(void* out, size_t at, const float* o, float f) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + at * 2);
#pragma unroll
    for (int v = 0; v < 4; ++v)
        dst[v] = make_uint4(pack2<QT>(o[8 * v + 0] * f, o[8 * v + 1] * f),
                            pack2<QT>(o[8 * v + 2] * f, o[8 * v + 3] * f),
                            pack2<QT>(o[8 * v + 4] * f, o[8 * v + 5] * f),
                            pack2<QT>(o[8 * v + 6] * f, o[8 * v + 7] * f));
}

// One sequence's new tokens, checked: false (and nothing to do) where they are
// inconsistent with the arrays.
__device__ __forceinline__ bool sequence(const Params& p, int s, int& q0, int& Ls, int& n) {
    q0 = p.query_start[s];
    const long long len = (long long)p.query_start[s + 1] - q0;
    n = p.context_lens[s];
    if (len < 0 || len > n || len > p.max_qlen || n > p.max_ctx ||
        (long long)n > (long long)p.MB * p.bs || q0 < 0 || q0 + len > p.T)
        return false;
    Ls = (int)len;
    return true;
}

template <int QT, bool FP8, int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(Plan<FP8, D>::THREADS, 1)
prefill_scored_kernel(const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const Params p) {
    using L = Plan<FP8, D>;
    constexpr int OT = FP8 ? (int)PA_F16 : QT;             // operand type
    constexpr int NSEG = L::NSEG, NS = L::NS, RS = L::RS;
    constexpr bool QCONV = FP8 && QT == PA_BF16;           // query rows brought to f16
    if (threadIdx.x < 3) prefetch_tensormap(threadIdx.x == 0 ? &tmq : threadIdx.x == 1 ? &tmk : &tmv);
    grid_dependency_wait();
    // grid (pair slots x key parts x kv heads, sequences, pair groups): adjacent
    // pairs of one (sequence, kv head) run side by side and share K / V through
    // L2; groups run longest first
    const int PG = p.pair_group;
    const int unit = (int)blockIdx.x / PG;
    const int pair = ((int)gridDim.z - 1 - (int)blockIdx.z) * PG + (PG - 1 - (int)blockIdx.x % PG);
    const int heads = p.Hq >> p.log2G;
    const int part = unit / heads, g = unit % heads;
    if (pair >= p.n_pairs) return;
    const int s = (int)blockIdx.y;
    int q0, Ls, n;
    if (!sequence(p, s, q0, Ls, n)) {
        if (pair == 0 && unit == 0 && threadIdx.x == 0) atomicOr(p.err, PA_DEV_BAD_CONTEXT);
        return;
    }
    const int c = n - Ls;                                  // tokens cached before this chunk
    const int iA = 2 * pair * p.TQ, iB = iA + p.TQ;
    if (iA >= Ls) return;
    const bool hasB = iB < Ls;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
    const uint32_t sb = smem_addr(sm);
    const uint32_t sQ = sb + L::Q, sOP = sb + L::OP, sRAW = sb + L::RAW;
    const uint32_t bar0 = sb + L::BAR;
    const uint32_t q_full = bar0, q_ready = bar0 + 8;
    auto full = [&](int i) { return bar0 + 8u * (2 + i); };
    auto free_ = [&](int i) { return bar0 + 8u * (2 + NS + i); };
    auto raw_full = [&](int i) { return bar0 + 8u * (2 + 2 * NS + i); };
    auto raw_free = [&](int i) { return bar0 + 8u * (2 + 2 * NS + RS + i); };
    const uint32_t bx = bar0 + 8u * (2 + 2 * NS + 2 * RS);
    auto s_full = [&](int x) { return bx + 8u * x; };
    auto p_full = [&](int x) { return bx + 8u * (2 + x); };
    auto pv_done = [&](int x) { return bx + 8u * (4 + x); };
    auto o_full = [&](int x) { return bx + 8u * (6 + x); };
    const uint32_t drain = bx + 64u, b_done = bx + 72u;
    auto turn = [&](int x, int w) { return bx + 80u + 8u * (4 * x + w); };
    volatile int* misc = reinterpret_cast<volatile int*>(sm + L::MISC);
    volatile int* abort_flag = misc + 1;
    int* dirty = reinterpret_cast<int*>(sm + L::MISC) + 2;     // first, last tile with zeroed values
    int* wr = reinterpret_cast<int*>(sm + L::MISC) + 4;        // 8 warps x Ranges
    volatile Stash* stash = reinterpret_cast<volatile Stash*>(sm + L::MISC + 144);
    float2* ml_b = reinterpret_cast<float2*>(sm + L::ML);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int x_row = warp < 4 || warp >= 8 || hasB ? warp >> 2 : 0;   // half whose row this thread has
    const int r = threadIdx.x & 127;
    const int it = (x_row == 1 ? iB : iA) + (r >> p.log2G);  // new token of this thread's row
    const bool row_ok = warp < 8 && it < Ls;
    const int pos = c + it;
    int lo = kNoLo, hi = kNoHi;
    if (row_ok) {
        lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        if (p.key_start) lo = max(lo, p.key_start[q0 + it]);
        hi = pos;
        if (p.prefix_lens) hi = max(hi, min(p.prefix_lens[s], n) - 1);
        if (lo > hi) lo = kNoLo, hi = kNoHi;
    }
    Ranges mine;                                           // of this warp's rows
    if (warp < 8) {
        mine.minlo = __reduce_min_sync(~0u, lo);
        mine.maxlo = __reduce_max_sync(~0u, row_ok ? lo : -1);
        mine.minhi = __reduce_min_sync(~0u, row_ok ? hi : INT_MAX);
        mine.maxhi = __reduce_max_sync(~0u, hi);
        if (lane == 0) {
            wr[4 * warp] = mine.minlo;
            wr[4 * warp + 1] = mine.maxlo;
            wr[4 * warp + 2] = mine.minhi;
            wr[4 * warp + 3] = mine.maxhi;
        }
    }
    if (threadIdx.x == 0) {
        const int users = hasB ? slot_halves(NS, true) : slot_halves(NS, false);
        mbar_init(q_full, 1);
        mbar_init(q_ready, hasB ? 256 : 128);
#pragma unroll 1
        for (int i = 0; i < NS; ++i) {
            mbar_init(full(i), FP8 ? 4 : 1);
            mbar_init(free_(i), users);
        }
#pragma unroll 1
        for (int i = 0; i < RS; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_free(i), 4);
        }
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(p_full(x), 128);
            mbar_init(pv_done(x), 1);
            mbar_init(o_full(x), 1);
        }
        mbar_init(drain, 2);
        mbar_init(b_done, 128);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) mbar_init(turn(i >> 2, i & 3), 1);
        misc[1] = 0;
        dirty[0] = INT_MAX;
        dirty[1] = -1;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(sb + L::MISC, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::MISC);

    // the halves' ranges, and which key tiles this CTA takes
    auto half = [&](int x) {
        Ranges q = {kNoLo, -1, INT_MAX, kNoHi};
#pragma unroll 1
        for (int w = 4 * x; w < 4 * x + 4; ++w) {
            q.minlo = min(q.minlo, wr[4 * w]);
            q.maxlo = max(q.maxlo, wr[4 * w + 1]);
            q.minhi = min(q.minhi, wr[4 * w + 2]);
            q.maxhi = max(q.maxhi, wr[4 * w + 3]);
        }
        return q;
    };
    const Ranges ra = half(0), rb = half(1);               // alike without B (its rows are A's)
    const int lo_c = min(ra.minlo, rb.minlo), hi_c = max(ra.maxhi, rb.maxhi);
    const int maxlo_c = max(ra.maxlo, rb.maxlo), minhi_c = min(ra.minhi, rb.minhi);
    const int kbase = hi_c < 0 ? 0 : lo_c & ~(p.bs - 1);
    const int all = hi_c < 0 ? 0 : (hi_c - kbase) / kBN + 1;   // key tiles of the pair
    const int parts = p.max_parts == 1 ? 1 : max(1, min(p.max_parts, (all + p.part_tiles - 1) / p.part_tiles));
    const int t0 = parts == 1 ? 0 : part * p.part_tiles;
    const int nt = part >= parts ? 0 : part == parts - 1 ? all - t0 : p.part_tiles;
    const int kb = kbase + t0 * kBN;                       // first key of tile 0
    const int hq = g * p.G + (r & (p.G - 1));              // query head of this thread's row
    const size_t out_row = (size_t)(q0 + it) * p.Hq + hq;

    const bool writes = row_ok && (hasB || warp < 4);
    if (nt == 0) {                                         // CTA-uniform: no key for any row
        if (writes && parts == 1 && part == 0) {
            const float zero[32] = {};
#pragma unroll 1
            for (int c4 = 0; c4 < D / 32; ++c4) store32<QT>(p.out, out_row * D + c4 * 32, zero, 0.f);
        }
        if (writes && p.max_parts > 1)
            p.ws_ml[out_row * p.max_parts + part] = make_float2(-INFINITY, parts == 1 && part == 0 ? -1.f : 0.f);
        __syncthreads();
        if (warp == 9) tmem_dealloc(tmem, kTmemCols);
        return;
    }
    // tiles [f, e) of a half hold keys its rows see; without B the halves take
    // the even and the odd tiles
    auto span = [&](const Ranges& q, int& f, int& e) {
        f = 0;
        e = nt;
        if (hasB) {
            f = max(0, (q.minlo - kb) >> 7);
            e = q.maxhi < kb ? 0 : min(nt, ((q.maxhi - kb) >> 7) + 1);
            if (q.maxhi < 0 || f >= e) f = e = 0;
        }
    };
    // some row of the CTA does not see all keys of tile j
    auto masked = [&](int j) { return kb + j * kBN < maxlo_c || kb + j * kBN + kBN - 1 > minhi_c; };

    if (threadIdx.x == 0) {
        stash->q0 = q0;
        stash->iA = iA;
        stash->g = g;
        stash->part = part;
        stash->parts = parts;
        stash->nt = nt;
        stash->kb = kb;
        stash->maxlo = maxlo_c;
        stash->minhi = minhi_c;
    }
    __syncthreads();
    auto tS = [&](int x) { return tmem + 256u * x; };
    auto tO = [&](int x) { return tmem + 256u * x + 128u; };
    // use u of the operand slots (K_j: u = 2j, V_j: u = 2j + 1)
    auto slot = [&](int u) { return u % NS; };
    auto phase = [&](int u) { return (uint32_t)(u / NS) & 1u; };

    if (warp == 8) {
        // ------------------------------------------------------------ copies
        regs_dec<L::ROTHER>();
        const int bpt = kBN >> p.log2bs;                       // blocks per key tile
        const uint32_t box = (uint32_t)p.bs * 128u;
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, (hasB ? 2 : 1) * L::TILE);
#pragma unroll 1
            for (int x = 0; x < (hasB ? 2 : 1); ++x)
#pragma unroll 1
                for (int sg = 0; sg < NSEG; ++sg)
                    tma_load_3d(sQ + x * L::TILE + sg * kSeg, &tmq, q_full, sg * 64, g * p.G,
                                q0 + (x ? iB : iA));
        }
        constexpr int RING = FP8 ? RS : NS;
        constexpr uint32_t TX = FP8 ? kSeg : L::TILE;
        int started = 0;
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
            const int lb = ((kb + j * kBN) >> p.log2bs) + lane;
            // a block past the last visible key, or an id outside the cache,
            // reads block NB: zeros
            int id = (int)p.NB;
            if (lane < bpt && (lb << p.log2bs) <= hi_c) {
                const int t = p.block_tables[(size_t)s * p.MB + lb];
                if (t >= 0 && (long long)t < p.NB) id = t;
                else atomicOr(p.err, PA_DEV_BAD_BLOCK);
            }
            bool ok = true;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int u = 2 * j + kv, st = u % RING;
                const uint32_t fb = FP8 ? raw_full(st) : full(st);
                ok = warp_wait(FP8 ? raw_free(st) : free_(st), ((u / RING) & 1) ^ 1, abort_flag, p.err,
                               10 + kv);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(fb, TX);
                __syncwarp();
                if (lane < bpt) {
                    if constexpr (FP8) {
                        tma_load_4d_plain(sRAW + st * kSeg + lane * box, kv ? &tmv : &tmk, fb, 0, g,
                                          0, id);
                    } else {
#pragma unroll 1
                        for (int sg = 0; sg < NSEG; ++sg)
                            tma_load_4d_plain(sOP + st * L::TILE + sg * kSeg + lane * box,
                                              kv ? &tmv : &tmk, fb, sg * 64, g, 0, id);
                    }
                }
                started = u + 1;
            }
            if (!ok) break;
        }
        // every copy this warp started has landed before the CTA may exit
#pragma unroll 1
        for (int i = 0; i < RING && i < started; ++i) {
            const int last = i + (started - 1 - i) / RING * RING;
            warp_wait(FP8 ? raw_full(i) : full(i), (last / RING) & 1, abort_flag, p.err, 17, false);
        }
        warp_wait(q_full, 0, abort_flag, p.err, 17, false);
    } else if (warp == 9 || warp == 10) {
        // -------------------------------------------------------------- MMAs
        regs_dec<L::ROTHER>();
        const int x = warp - 9;
        constexpr int ABF = OT == PA_BF16 ? 1 : 0;
        const uint32_t id_s = idesc_f16(ABF, 0, kBN), id_o = idesc_f16(ABF, 1, D);
        const uint32_t qb = sQ + (hasB ? x : 0) * L::TILE;
        int f, e;
        span(x ? rb : ra, f, e);
        // the last tile this half takes part in
        const int last = hasB ? e - 1 : nt - 1 - ((nt - 1 - x) & 1);
        bool ok = warp_wait(QCONV ? q_ready : q_full, 0, abort_flag, p.err, 7);
        int i = 0;                                             // tiles done
#pragma unroll 1
        for (int j = 0; j < nt && ok; ++j) {
            const bool act = j >= f && j < e;
            const int sk = slot(2 * j), sv = slot(2 * j + 1);
            if (!hasB && (j & 1) != x) {
                // The other half's tile.  Waits go by the parity of a slot's phase, so
                // where the halves' tiles share slots a warp sees the phases of both, and
                // a slot is filled again only after both have: one that skipped a phase,
                // or looked late, would take an old one for its own.
                if constexpr (slot_halves(NS, false) == 2) {
                    ok = warp_wait(full(sk), phase(2 * j), abort_flag, p.err, 8);
                    if (ok && lane == 0) mbar_arrive(free_(sk));
                    ok = ok && warp_wait(full(sv), phase(2 * j + 1), abort_flag, p.err, 9);
                    if (ok && lane == 0) mbar_arrive(free_(sv));
                }
                continue;
            }
            if (!(ok = warp_wait(full(sk), phase(2 * j), abort_flag, p.err, 8))) break;
            tc_fence_after();
            if (lane == 0) {
                if (act) {
                    // low descriptor word: address / 16 | leading offset / 16 << 16
                    const uint32_t hi32 = (uint32_t)(sdesc(0, 16) >> 32);
                    const uint32_t alo = (qb >> 4) | (1u << 16);
                    const uint32_t blo = ((sOP + sk * L::TILE) >> 4) | (1u << 16);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kSeg + (kk & 3) * 32) >> 4;
                        tc_mma_lh(tS(x), alo + off, hi32, blo + off, hi32, id_s, kk > 0);
                    }
                    tc_commit(s_full(x));
                    tc_commit(free_(sk));
                } else {
                    mbar_arrive(free_(sk));                    // this half does not read it
                }
            }
            __syncwarp();
            if (!(ok = warp_wait(full(sv), phase(2 * j + 1), abort_flag, p.err, 9))) break;
            if (act) {
                if (!FP8 && masked(j)) {
                    // with B both warps look at (and mend) the whole tile, alike
                    const uint32_t tile = sOP + sv * L::TILE + lane * 16;
                    bool bad = false;
#pragma unroll 8
                    for (int v = 0; v < L::TILE; v += 512) bad |= nonfinite<OT>(lds128(tile + v));
                    if (__any_sync(~0u, bad)) {
                        // marked first: the other warp may find the tile mended already
                        if (lane == 0) {
                            atomicMin(dirty, j);
                            atomicMax(dirty + 1, j);
                            __threadfence_block();
                        }
                        __syncwarp();
#pragma unroll 1
                        for (int v = 0; v < L::TILE; v += 512) sts128(tile + v, finite_only<OT>(lds128(tile + v)));
                    }
                    fence_proxy_async_smem();                  // this warp's mending, or what it saw of the other's
                    __syncwarp();
                }
                if (!(ok = warp_wait(p_full(x), i & 1, abort_flag, p.err, 13))) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t vhi = (uint32_t)(sdesc(0, kSeg) >> 32);
                    const uint32_t vlo = ((sOP + sv * L::TILE) >> 4) | ((uint32_t)(kSeg >> 4) << 16);
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        tc_mma_ts_lh(tO(x), tS(x) + kk * 8, vlo + kk * 128, vhi, id_o,
                                     (i > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(pv_done(x));
                    if (j == last) tc_commit(o_full(x));
                    tc_commit(free_(sv));
                }
                ++i;
            } else if (lane == 0) {
                mbar_arrive(free_(sv));
            }
            __syncwarp();
        }
        // every MMA this warp issued completes before tensor memory is freed
        if (lane == 0) tc_commit(drain);
        __syncwarp();
        warp_wait(drain, 0, abort_flag, p.err, 16, false);
    } else if (warp == 11) {
        regs_dec<L::ROTHER>();
    } else if (warp >= 12) {
        // ------------------------------------------- E4M3 codes to f16 operands
        regs_dec<L::ROTHER>();
        if constexpr (FP8) {
            const int tid = threadIdx.x - 384;
#pragma unroll 1
            for (int u = 0; u < 2 * nt; ++u) {
                const int rs = u % RS, st = slot(u);
                if (!warp_wait(raw_full(rs), (u / RS) & 1, abort_flag, p.err, 9)) break;
                if (!warp_wait(free_(st), phase(u) ^ 1, abort_flag, p.err, 10)) break;
                const uint32_t src = sRAW + rs * kSeg, dst = sOP + st * L::TILE;
                const bool look = (u & 1) && masked(u >> 1);
                bool bad = false;
#pragma unroll 4
                for (int i = tid; i < kBN * 8; i += 128) {
                    // 16 codes of row t: chunk ch of the row, two chunks of the
                    // operand segment ch / 4.  The lanes of segment 1 write their
                    // two in the other order, so a store meets every bank once.
                    const int t = i >> 3, ch = i & 7;
                    const uint4 w = lds128(src + swz128(t, ch));
                    const uint2 h0 = widen(w.x), h1 = widen(w.y), h2 = widen(w.z), h3 = widen(w.w);
                    const uint4 a = make_uint4(h0.x, h0.y, h1.x, h1.y), b = make_uint4(h2.x, h2.y, h3.x, h3.y);
                    if (look) bad |= nonfinite<PA_F16>(a) | nonfinite<PA_F16>(b);
                    const uint32_t seg = dst + (ch >> 2) * kSeg;
                    const int oc = 2 * (ch & 3), sw = ch >> 2;
                    sts128(seg + swz128(t, oc + sw), sw ? b : a);
                    sts128(seg + swz128(t, oc + 1 - sw), sw ? a : b);
                }
                if (bad) {                                   // this thread's chunks once more
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        const int t = (tid >> 3) + 16 * (i >> 1), ch = tid & 7;
                        const uint32_t at = dst + (ch >> 2) * kSeg + swz128(t, 2 * (ch & 3) + (i & 1));
                        sts128(at, finite_only<PA_F16>(lds128(at)));
                    }
                    atomicMin(dirty, u >> 1);
                    atomicMax(dirty + 1, u >> 1);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full(st));
                    mbar_arrive(raw_free(rs));
                }
            }
        }
    } else {
        // ----------------------------------------- softmax (rows of half X)
        regs_inc<L::RSOFT>();
        const int x = warp >> 2;
        const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
        int f, e;
        span(x ? rb : ra, f, e);
        const int first = hasB ? f : x, step = hasB ? 1 : 2, end = hasB ? e : nt;
        float m_use = -INFINITY, lsum = 0.f;
        bool ok = true;
        float sl = p.sl;
        if constexpr (QCONV) {
            float* rowscale = reinterpret_cast<float*>(sm + L::ROWSCALE);
            ok = warp_wait(q_full, 0, abort_flag, p.err, 7);
            if (ok && (hasB || x == 0)) {
                rowscale[threadIdx.x] = row_to_f16<D>(sQ + x * L::TILE, r);
                fence_proxy_async_smem();
                mbar_arrive(q_ready);
            }
            ok = ok && warp_wait(q_ready, 0, abort_flag, p.err, 7);
            if (ok) sl *= rowscale[hasB ? threadIdx.x : r];
        }
        // a factor that fp32 rounds to 0: the scores are 0, and masked ones are to stay -inf
        sl = fmaxf(sl, __int_as_float(1));
        const float slope = BIAS && row_ok ? p.slopes[hq] * kLog2e : 0.f;
        // distances by the difference alone (no keys of a prefix ahead of a row), whose
        // products lose nothing that matters
        const bool linear = BIAS && !p.prefix_lens && __all_sync(~0u, fabsf(slope) <= 64.f);
        const bool live = __any_sync(~0u, row_ok);         // a warp without rows only keeps step
        // tiles [ja, jb) need no mask in this warp
        const int ja = mine.maxlo <= kb ? 0 : ((min(mine.maxlo, INT_MAX - kBN) - kb - 1) >> 7) + 1;
        const int jb = mine.minhi == INT_MAX ? INT_MAX : mine.minhi < kb ? 0 : (mine.minhi - kb + 1) >> 7;
        // The turns: tiles [jt, jt + nturn) of A and B alternate (without B the
        // even and the odd tiles), where this warp and its partner both have rows.
        int jt = first, nturn = nt / 2;
        if (hasB) {
            int fo, eo;
            span(x ? ra : rb, fo, eo);
            jt = max(f, fo);
            const bool partner = iB + (((warp & 3) * 32) >> p.log2G) < Ls;
            nturn = partner ? min(e, eo) - jt : 0;
        }
        const uint32_t my_turn = turn(x, warp & 3), next_turn = turn(x ^ 1, warp & 3);
        int i = 0;                                         // tiles done
#pragma unroll 1
        for (int j = first; j < end && ok; j += step, ++i) {
            if (!(ok = warp_wait(s_full(x), i & 1, abort_flag, p.err, 12))) break;
            if (!live) {
                mbar_arrive(p_full(x));
                continue;
            }
            tc_fence_after();
            const bool mask = j < ja || j >= jb;
            const int k0 = kb + j * kBN;
            const float2 sl2 = make_float2(sl, sl);
            const uint32_t ts = tS(x) + lrow;
            float tmax = -INFINITY;
            // Scores without a cap stay in registers, a row of 128.  With one the code of
            // a tile would be three times as long, and instructions of straight code
            // arrive at half the rate they can be issued: capped scores are worked on 32
            // columns at a time, in rolled loops from tensor memory and back (chunked
            // prefill, capped: 1692 -> 1497 us, 1537 with all that came later; without: 1257
            // against 1295, with a bias 1654 against 1689).
            float sv[CAP ? 1 : kBN], s[CAP ? 32 : 1];
            int fit = 0;                   // terms: S keeps the products, and the cap is taken below
            if constexpr (!CAP) {
#pragma unroll
                for (int c4 = 0; c4 < kBN / 32; ++c4) tmem_ld32(ts + c4 * 32, sv + c4 * 32);
                tmem_wait_ld();
                if constexpr (BIAS) {
                    const float d0 = (float)(pos - k0);        // distance of key 0
                    if (linear) {
                        const float b0 = -slope * d0;
#pragma unroll
                        for (int k = 0; k < kBN; k += 2) {
                            const float2 z = fma2(make_float2(sv[k], sv[k + 1]), sl2,
                                                  make_float2(fmaf(slope, (float)k, b0), fmaf(slope, (float)(k + 1), b0)));
                            sv[k] = z.x;
                            sv[k + 1] = z.y;
                        }
                    } else {
                        // distances as exact small integers (|i - p|: keys of a prefix
                        // ahead of the row; slopes whose products lose what matters)
#pragma unroll
                        for (int k = 0; k < kBN; ++k) sv[k] = fmaf(-slope, fabsf(d0 - (float)k), sv[k] * sl);
                    }
                }
                // keys outside a row's range become -inf; a tile that no row of the
                // warp masks skips the compares
                if (mask) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t bits = range_word(lo == kNoLo ? kBN : lo - k0, hi - k0, w);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(bits & (1u << k))) sv[32 * w + k] = -INFINITY;
                    }
                }
                // row maximum as 8 independent chains of three-input maxima
                float pm[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) pm[k] = sv[k];
#pragma unroll
                for (int k = 8; k < kBN; k += 2) pm[(k >> 1) & 7] = max3(pm[(k >> 1) & 7], sv[k], sv[k + 1]);
                tmax = fmaxf(max3(pm[0], pm[1], pm[2]), fmaxf(max3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])));
                if constexpr (!BIAS) tmax *= sl;               // scale > 0
            } else {
                // With a cap u = 4 scale x / softcap (the factor sl), and the score is
                // cap_log2 * tanh(u / 4) in log2 units.  `fit`: no |u| of the warp exceeds
                // 2 (4) and no row masks; the four-term (six-term) fit then runs with the
                // exponentials below, and the row's maximum is the same fit of its largest u
                // (another form of the tanh would be off by 2^-23 of the cap, which for a cap
                // of 1e9 is more than the probabilities' range).
                // Else the modified and masked scores go back into S, each by its own size: on a
                // tile that some row masks a vote would let keys that a row does not see choose
                // its form.  (8 x 2048 queries of
                // scale 3: cap 15, mostly above 2, 2110 us with the four-term fit alone and
                // 1650 with both; caps 30 and 50, nearly all below 2, 1507 and 1497 us
                // against 1525 and 1530, for the code that they pass over.  A score's own
                // size in place of the vote on masked tiles: 1684, 1530 and 1537; cap 10,
                // mostly above 4, 2748 -> 2933.)
                if (!BIAS && !mask) {
                    float lo32 = INFINITY;
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; ++c4) {
                        tmem_ld32(ts + c4 * 32, s);
                        tmem_wait_ld32(s);
                        tmax = fmaxf(tmax, max32(s));
                        lo32 = fminf(lo32, min32(s));
                    }
                    // (rows there are not have no part in the choice)
                    const float top = row_ok ? fmaxf(fabsf(tmax), fabsf(lo32)) * sl : 0.f;
                    fit = !__any_sync(~0u, !(top <= 2.f)) ? 4 : !__any_sync(~0u, !(top <= 4.f)) ? 6 : 0;
                }
                if (fit) {
                    tmax = fitted(tmax * sl, p.cap_log2, fit);
                } else {
                    // modified and masked scores back into S
                    tmax = -INFINITY;
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; ++c4) {
                        tmem_ld32(ts + c4 * 32, s);
                        tmem_wait_ld32(s);
                        const float cl = p.cap_log2;
                        auto capped = [&](auto far) {
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                const float2 z = capped2<decltype(far)::value>(mul2(make_float2(s[k], s[k + 1]), sl2), cl);
                                s[k] = z.x;
                                s[k + 1] = z.y;
                            }
                        };
                        if (__any_sync(~0u, fmaxf(max32(s), -min32(s)) * sl > 4.f)) capped(std::true_type());
                        else capped(std::false_type());
                        if constexpr (BIAS) {
                            const float d0 = (float)(pos - (k0 + c4 * 32));      // distance of the first key
                            if (linear) {
                                const float b0 = -slope * d0;
#pragma unroll
                                for (int k = 0; k < 32; k += 2) {
                                    const float2 b = make_float2(fmaf(slope, (float)k, b0), fmaf(slope, (float)(k + 1), b0));
                                    const float2 z = add2(make_float2(s[k], s[k + 1]), b);
                                    s[k] = z.x;
                                    s[k + 1] = z.y;
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    s[k] = fmaf(-slope, fabsf(d0 - (float)k), s[k]);
                            }
                        }
                        if (mask) {
                            const uint32_t bits = range_word(lo == kNoLo ? kBN : lo - k0, hi - k0, c4);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(bits & (1u << k))) s[k] = -INFINITY;
                        }
                        tmax = fmaxf(tmax, max32(s));
                        tmem_st32(ts + c4 * 32, s);
                    }
                    tmem_wait_st();
                }
            }
            const float m_new = fmaxf(m_use, tmax);
            const bool raise = m_new > m_use + kRescaleLog2;
            const float alpha = raise ? ex2(m_use - m_new) : 1.f;
            if (raise) m_use = m_new;
            lsum *= alpha;
            if (i > 0 && __any_sync(~0u, raise)) {
                // O_X holds P.V of the tiles before once the last of them completes
                if (!(ok = warp_wait(pv_done(x), (i - 1) & 1, abort_flag, p.err, 14))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c4 = 0; c4 < D / 32; ++c4) {
                    float o[32];
                    tmem_ld32(tO(x) + lrow + c4 * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int v = 0; v < 32; ++v) o[v] *= alpha;
                    tmem_st32(tO(x) + lrow + c4 * 32, o);
                }
                tmem_wait_st();
            }
            // probabilities, rounded to the operand type, two per 32-bit column
            // over the scores they came from; a row that has seen no key yet has
            // no maximum to take off.  f16 operands are 2^7 times as large (at most
            // 2^15), so that small ones keep their bits; l carries the same factor.
            const float nm = (OT == PA_F16 ? 7.f : 0.f) - (m_use == -INFINITY ? 0.f : m_use);
            const float2 nm2 = make_float2(nm, nm);
            if constexpr (BIAS && !CAP) {
#pragma unroll
                for (int k = 0; k < kBN; k += 2) {
                    const float2 d = add2(make_float2(sv[k], sv[k + 1]), nm2);
                    sv[k] = d.x;
                    sv[k + 1] = d.y;
                }
            }
            const int at = hasB ? j - jt : i;                  // this tile's turn
            if (x ? at >= 0 && at < nturn : at > 0 && at <= nturn)
                if (!(ok = warp_wait(my_turn, (at - 1 + x) & 1, abort_flag, p.err, 18))) break;
            float2 sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
            if constexpr (!CAP) {
#pragma unroll
                for (int c16 = 0; c16 < kBN / 32; ++c16) {
                    uint32_t w[16];
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int k = c16 * 32 + 2 * v;
                        const float2 z = make_float2(sv[k], sv[k + 1]);
                        const float2 d = BIAS ? z : fma2(z, sl2, nm2);
                        sv[k] = ex2(d.x);
                        sv[k + 1] = ex2(d.y);
                        w[v] = pack2<OT>(sv[k], sv[k + 1]);
                    }
                    tmem_st16(ts + c16 * 16, w);
                }
            } else {
                // two chunks a round, the next one on its way while one is worked on
                float s2[32];
                auto chunk = [&](int c4, float* s, auto arg) {
                    uint32_t w[16];
                    arg(s);
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        s[2 * v] = ex2(s[2 * v]);
                        s[2 * v + 1] = ex2(s[2 * v + 1]);
                        w[v] = pack2<OT>(s[2 * v], s[2 * v + 1]);
                        sum[v & 1] = add2(sum[v & 1], make_float2(s[2 * v], s[2 * v + 1]));
                    }
                    tmem_st16(ts + c4 * 16, w);
                };
                auto chunks = [&](auto arg) {
                    tmem_ld32(ts, s);
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; c4 += 2) {
                        tmem_wait_ld32(s);
                        tmem_ld32(ts + c4 * 32 + 32, s2);
                        chunk(c4, s, arg);
                        tmem_wait_ld32(s2);
                        if (c4 == 0) tmem_ld32(ts + 64, s);
                        chunk(c4 + 1, s2, arg);
                    }
                };
                if (!BIAS && fit == 4) {
                    const float cl = p.cap_log2;
                    float2 co[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) co[t] = make_float2(kTanh4[t] * cl, kTanh4[t] * cl);
                    chunks([&](float* s) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 u = mul2(make_float2(s[k], s[k + 1]), sl2), v = mul2(u, u);
                            const float2 d = fma2(u, fma2(fma2(fma2(co[3], v, co[2]), v, co[1]), v, co[0]), nm2);
                            s[k] = d.x;
                            s[k + 1] = d.y;
                        }
                    });
                } else if (!BIAS && fit) {
                    const float cl = p.cap_log2;
                    float2 co[6];
#pragma unroll
                    for (int t = 0; t < 6; ++t) co[t] = make_float2(kTanh6[t] * cl, kTanh6[t] * cl);
                    chunks([&](float* s) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 u = mul2(make_float2(s[k], s[k + 1]), sl2), v = mul2(u, u);
                            float2 y = co[5];
#pragma unroll
                            for (int t = 4; t >= 0; --t) y = fma2(y, v, co[t]);
                            const float2 d = fma2(u, y, nm2);
                            s[k] = d.x;
                            s[k + 1] = d.y;
                        }
                    });
                } else {
                    chunks([&](float* s) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 d = add2(make_float2(s[k], s[k + 1]), nm2);
                            s[k] = d.x;
                            s[k + 1] = d.y;
                        }
                    });
                }
            }
            if (at >= 0 && at < nturn) {
                __syncwarp();
                if (lane == 0) mbar_arrive(next_turn);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(p_full(x));
            // without a cap the row sum is not on the way to P.V: it is taken after the hand-off
            if constexpr (!CAP) {
#pragma unroll
                for (int k = 0; k < kBN; k += 2)
                    sum[(k >> 1) & 3] = add2(sum[(k >> 1) & 3], make_float2(sv[k], sv[k + 1]));
            }
            lsum += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
                    ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
        }
        // -------------------------------------------------------- epilogue
        float fa = 1.f, fb = 0.f;                          // weights of O_X and O_B
        const bool has_o = i > 0;                          // the half's O was written
        if (ok && has_o) ok = warp_wait(o_full(x), 0, abort_flag, p.err, 15);
        if (p.max_parts > 1) launch_dependents();              // the join may start launching
        const int ntiles = stash->nt;
        if (!hasB) {
            if (x == 1) {
                ml_b[r] = make_float2(m_use, lsum);
                mbar_arrive(b_done);
                ok = false;                                // half A writes the rows
            } else if (ok && ntiles > 1) {
                ok = warp_wait(b_done, 0, abort_flag, p.err, 20) &&
                     warp_wait(o_full(1), 0, abort_flag, p.err, 15);
                const float2 b = ml_b[r];
                const float m = fmaxf(m_use, b.x);
                const float base = m == -INFINITY ? 0.f : m;
                fa = ex2(m_use - base);
                fb = ex2(b.x - base);
                lsum = lsum * fa + b.y * fb;
                m_use = m;
            }
        }
        if (ok && live) {
            tc_fence_after();
            const int g = stash->g, part = stash->part, kb = stash->kb;
            const int it = stash->iA + (hasB && x ? p.TQ : 0) + (r >> p.log2G);
            const size_t out_row = (size_t)(stash->q0 + it) * p.Hq + g * p.G + (r & (p.G - 1));
            const bool record = stash->parts > 1;
            const float inv = record ? 1.f : lsum == 0.f ? 0.f : p.v_scale / lsum;
            const bool fix = dirty[1] >= 0;                // values were taken out of V
            const bool both = !hasB && ntiles > 1;
#pragma unroll 1
            for (int c4 = 0; c4 < D / 32; ++c4) {
                float o[32];
                if (has_o) {
                    tmem_ld32(tO(x) + lrow + c4 * 32, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int v = 0; v < 32; ++v) o[v] = 0.f;
                }
                if (both) {
                    float ob[32];
                    tmem_ld32(tO(1) + lrow + c4 * 32, ob);
                    tmem_wait_ld();
#pragma unroll
                    for (int v = 0; v < 32; ++v) o[v] = o[v] * fa + ob[v] * fb;
                }
                if (fix && row_ok && lo != kNoLo) {
                    const int ka = max(lo, kb + dirty[0] * kBN);
                    const int kz = min(hi, kb + dirty[1] * kBN + kBN - 1);
#pragma unroll 1
                    for (int k = ka; k <= kz; ++k) {
                        const int k0 = k - ((k - kb) & (kBN - 1));
                        if (k0 >= stash->maxlo && k0 + kBN - 1 <= stash->minhi) {
                            k = k0 + kBN - 1;              // this tile kept its values
                            continue;
                        }
                        const int id = p.block_tables[(size_t)s * p.MB + (k >> p.log2bs)];
                        if (id < 0 || (long long)id >= p.NB) continue;
                        const size_t at = (((size_t)id * p.bs + (k & (p.bs - 1))) * (p.Hq / p.G) + g) * D + c4 * 32;
#pragma unroll
                        for (int v = 0; v < 32; ++v) {
                            const float y = cache_value<FP8 ? (int)PA_FP8_E4M3 : QT>(p.v_cache, at + v);
                            if (!isfinite(y)) o[v] += y;
                        }
                    }
                }
                if (row_ok) {
                    if (record) {
                        float4* dst = reinterpret_cast<float4*>(p.ws_o + (out_row * p.max_parts + part) * D + c4 * 32);
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            dst[v] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                    } else {
                        store32<QT>(p.out, out_row * D + c4 * 32, o, inv);
                    }
                }
            }
            // l = -1 marks a row that needs no join
            if (row_ok && p.max_parts > 1)
                p.ws_ml[out_row * p.max_parts + part] = make_float2(m_use, record ? lsum : -1.f);
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Join of the key parts: one warp per (new token, query head) row.  Nothing but
// latencies bounds it: the lengths are read while the attention kernel ends (its
// CTAs let this grid start after their own wait for the kernels before), a row's
// maxima and sums in one load of a part a lane, and eight records at a time (4 new
// tokens on 30000 in 17 parts, both kernels: 30.8 us before, 28.2).
template <int QT, int D>
__global__ void __launch_bounds__(256) prefill_scored_merge(const Params p) {
    const int s = (int)blockIdx.y, lane = threadIdx.x & 31;
    int q0, Ls, n;
    const bool good = sequence(p, s, q0, Ls, n);
    grid_dependency_wait();
    if (!good) return;
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (long long)Ls * p.Hq) return;
    const size_t row = (size_t)q0 * p.Hq + (size_t)w;
    const float2* ml = p.ws_ml + row * p.max_parts;
    float2 part = lane < p.max_parts ? ml[lane] : make_float2(-INFINITY, 0.f);
    if (__shfl_sync(~0u, part.y, 0) == -1.f) return;       // written by the attention kernel
    float m = part.x;
#pragma unroll 1
    for (int i = 32 + lane; i < p.max_parts; i += 32) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    constexpr int E = D / 32, kAhead = 8;
    float acc[E] = {}, l = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < p.max_parts; i0 += kAhead) {
        if (i0 && (i0 & 31) == 0) part = i0 + lane < p.max_parts ? ml[i0 + lane] : make_float2(-INFINITY, 0.f);
        float sum[kAhead], v[kAhead][E];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            sum[j] = __shfl_sync(~0u, part.y, (i0 + j) & 31);
            if (sum[j] == 0.f) continue;                   // no key seen: nothing was written
            const float* o = p.ws_o + (row * p.max_parts + i0 + j) * D + lane * E;
            if constexpr (E == 4) {
                const float4 x = *reinterpret_cast<const float4*>(o);
                v[j][0] = x.x;
                v[j][1] = x.y;
                v[j][2] = x.z;
                v[j][3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2*>(o);
                v[j][0] = x.x;
                v[j][1] = x.y;
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const float f = ex2(__shfl_sync(~0u, part.x, (i0 + j) & 31) - base);
            if (sum[j] == 0.f) continue;
            l += sum[j] * f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(v[j][e], f, acc[e]);
        }
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * (size_t)(D * 2)) + lane * (E / 2);
    dst[0] = pack2<QT>(acc[0] * inv, acc[1] * inv);
    if constexpr (E == 4) dst[1] = pack2<QT>(acc[2] * inv, acc[3] * inv);
}

template <int QT, bool FP8, int D, bool CAP, bool BIAS>
cudaError_t launch_one(const Launch& a) {
    using L = Plan<FP8, D>;
    auto kern = prefill_scored_kernel<QT, FP8, D, CAP, BIAS>;
    cudaError_t e = ensure_dynamic_smem<prefill_scored_kernel<QT, FP8, D, CAP, BIAS>>(L::BYTES);
    if (e != cudaSuccess) return e;
    // the register split waits for registers the block must have been given
    static std::atomic<int> regs{0};
    int have = regs.load(std::memory_order_relaxed);
    if (!have) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
        have = (fa.numRegs + 7) / 8 * 8;
        regs.store(have, std::memory_order_relaxed);
    }
    if (have * L::THREADS < L::RTOTAL) return cudaErrorInvalidConfiguration;
    return launch_pdl(kern, a.grid, dim3(L::THREADS), (size_t)L::BYTES, a.stream, *a.mq, *a.mk, *a.mv, *a.p);
}

template <int QT, int D> cudaError_t launch_merge(const Launch& a) {
    if (a.p->max_parts == 1) return cudaSuccess;
    const unsigned rows = (unsigned)(((long long)a.p->max_qlen * a.p->Hq + 7) / 8);
    return launch_pdl(prefill_scored_merge<QT, D>, dim3(rows, a.grid.y), dim3(256), 0, a.stream, *a.p);
}

template <int QT, bool FP8, int D>
cudaError_t launch_mod(const Launch& a) {
    const bool cap = a.p->cap_log2 > 0.f, bias = a.p->slopes != nullptr;
    cudaError_t e;
    if (cap) e = bias ? launch_one<QT, FP8, D, true, true>(a) : launch_one<QT, FP8, D, true, false>(a);
    else e = bias ? launch_one<QT, FP8, D, false, true>(a) : launch_one<QT, FP8, D, false, false>(a);
    return e == cudaSuccess ? launch_merge<QT, D>(a) : e;
}

}  // namespace ps
