// Chunk attention with modified scores for few query rows (pa_prefill_scored,
// at most 32 rows of a kv head: L new tokens x G query heads), bound by the read
// of the cache.
//
// With few rows the roles of keys and queries are exchanged, so that the 128 rows
// of the MMA are keys and the few queries its columns:
//     S_j^T = K_j Q^T    128 keys x NR rows, one key per softmax thread
//     O^T  += V_j^T P_j^T   D x NR, V the MN-major A operand, P written to shared
//                        memory in the layout of V
// A softmax thread has 16 scores instead of 128, eight warps share the
// exponentials of a tile, and the next scores are computed meanwhile (S_j^T takes
// NR columns, so two fit).  The price is that a row's maximum lies across
// threads.  It is not needed every tile: scores are taken against the running
// reference m of their row, and only when one exceeds it by more than 8 (in log2
// units; the first tile always) the rows' four warps find the tile's maxima (a warp
// reduction a row) and rescale the rows that do.  A row's sum is kept per thread and added
// up once.
//
// 8-bit cache: four more warps widen the codes to f16 (exactly): K to tensor
// memory, from where the MMA takes it as its A operand, so it does not pass
// through shared memory again; V to shared memory.  Per 128-key tile of D = 128
// shared memory then moves 256 cycles' worth of arriving codes, 256 read back, 256
// of V written and 256 read by the MMA, and P; HBM brings the tile's 32 KB in
// 1400 cycles an SM.  A bf16 query row is scaled as in the kernel for many rows.
//
// Warps: four softmax warps for every 16 rows; then one for the copies, one for the
// MMAs of S^T, one for those of O^T, one idle; 8-bit: four for the widening.
// Tensor memory: O^T from 0, S^T from 32 and 64, K operands from 128 and 192.
// Waits are bounded and non-finite values handled as in the kernel for many rows.
#pragma once

#include "prefill_scored.cuh"

namespace ps {

template <bool FP8, int D, int NR>
struct FewPlan {
    static constexpr int NSEG = D / 64;
    static constexpr int TILE = NSEG * kSeg;
    // Operand slots: 16-bit a ring of KS K tiles and one of VS V tiles, 8-bit V tiles
    // and a ring of codes.  Every slot has one warp that waits for it: a wait goes by
    // the parity of the slot's phase, which a warp that skips a phase of it can mistake
    // for the one before (K and V in one ring of five did, and released slots under
    // copies in flight).
    static constexpr int KS = FP8 ? 0 : D == 64 ? 5 : 3, VS = FP8 ? 2 : D == 64 ? 5 : 2;
    static constexpr int NS = KS + VS;
    static constexpr int RS = FP8 ? 6 : 0;
    static constexpr int NG = NR / 16;                  // softmax warpgroups, 16 rows each
    static constexpr int QB = NR * 128 * NSEG;
    static constexpr int Q = 0;
    static constexpr int OP = QB;
    static constexpr int RAW = OP + NS * TILE;
    static constexpr int P = RAW + RS * kSeg;           // 2 x 128 keys x 128 bytes
    static constexpr int META = P + 2 * kSeg;
    // rows: lo, hi, position behind the cached tokens, slope, factor of their scores,
    // reference, alpha, sum
    static constexpr int METAB = NR * 4 * 8;
    // rows of values by thread, for what goes across threads
    static constexpr int XCH = META + METAB;
    static constexpr int XROW = 132 * 4;                // 128 values; rows 16 bytes apart in banks
    static constexpr int BAR = XCH + NR * XROW;
    // q_full, q_ready, full[NS], free[NS], raw_full[RS], raw_free[RS], k_full[2],
    // k_free[2], s_full[2], s_free[2], p_full[2], pv_done[2], sync[2], drain
    static constexpr int NBAR = 2 + 2 * NS + 2 * RS + 12 + 3;
    static constexpr int MISC = BAR + NBAR * 8;         // tensor memory, abort, dirty, ranges, flags
    static constexpr int BYTES = MISC + 64 + 1024;
    static_assert(BYTES <= 232448, "shared memory of one CTA");
    static constexpr int THREADS = 128 * (NG + 1 + (FP8 ? 1 : 0));
};

constexpr float kNoMax = -3e38f;      // reference of a row that has seen no key

// The largest of the warp's values, in every lane (NaN is passed over).
__device__ __forceinline__ float warp_max(float v) {
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

template <int QT, bool FP8, int D, int NR, bool CAP, bool BIAS>
__global__ void __launch_bounds__(FewPlan<FP8, D, NR>::THREADS, 1)
prefill_few_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const Params p) {
    using L = FewPlan<FP8, D, NR>;
    constexpr int OT = FP8 ? (int)PA_F16 : QT;
    constexpr int NSEG = L::NSEG, NS = L::NS, RS = L::RS, KS = L::KS, VS = L::VS;
    constexpr bool QCONV = FP8 && QT == PA_BF16;
    constexpr float SHIFT = OT == PA_F16 ? 7.f : 0.f;      // as in the kernel for many rows
    if (threadIdx.x < 3) prefetch_tensormap(threadIdx.x == 0 ? &tmq : threadIdx.x == 1 ? &tmk : &tmv);
    grid_dependency_wait();
    const int heads = p.Hq >> p.log2G;                         // heads of a part side by side
    const int part = (int)blockIdx.x / heads, g = (int)blockIdx.x % heads;
    const int s = (int)blockIdx.y;
    int q0, Ls, n;
    if (!sequence(p, s, q0, Ls, n)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, PA_DEV_BAD_CONTEXT);
        return;
    }
    if (Ls == 0) return;
    const int c = n - Ls;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
    const uint32_t sb = smem_addr(sm);
    const uint32_t bar0 = sb + L::BAR;
    const uint32_t q_full = bar0, q_ready = bar0 + 8;
    auto full = [&](int i) { return bar0 + 8u * (2 + i); };
    auto free_ = [&](int i) { return bar0 + 8u * (2 + NS + i); };
    auto raw_full = [&](int i) { return bar0 + 8u * (2 + 2 * NS + i); };
    auto raw_free = [&](int i) { return bar0 + 8u * (2 + 2 * NS + RS + i); };
    const uint32_t bx = bar0 + 8u * (2 + 2 * NS + 2 * RS);
    auto k_full = [&](int b) { return bx + 8u * b; };
    auto k_free = [&](int b) { return bx + 8u * (2 + b); };
    auto s_full = [&](int b) { return bx + 8u * (4 + b); };
    auto s_free = [&](int b) { return bx + 8u * (6 + b); };
    auto p_full = [&](int b) { return bx + 8u * (8 + b); };
    auto pv_done = [&](int b) { return bx + 8u * (10 + b); };
    auto sync = [&](int q) { return bx + 96u + 8u * q; };
    const uint32_t drain = bx + 112u;
    volatile int* misc = reinterpret_cast<volatile int*>(sm + L::MISC);
    volatile int* abort_flag = misc + 1;
    int* dirty = reinterpret_cast<int*>(sm + L::MISC) + 2;     // first, last tile with zeroed values
    int* ranges = reinterpret_cast<int*>(sm + L::MISC) + 4;    // lo, hi, largest lo, smallest hi
    volatile int* flags = misc + 8;                            // [group][2]: tile + 1 to raise in
    int* m_lo = reinterpret_cast<int*>(sm + L::META);
    int* m_hi = m_lo + NR;
    float* m_pos = reinterpret_cast<float*>(m_lo + 2 * NR);
    float* m_slope = m_pos + NR;
    float* m_scale = m_pos + 2 * NR;
    float* m_nm = m_pos + 3 * NR;                              // SHIFT - reference
    float* m_alpha = m_pos + 4 * NR;
    float* m_sum = m_pos + 5 * NR;

    constexpr int NG = L::NG, W0 = 4 * NG;                     // W0: the first warp that is no softmax one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const int it = lane >> p.log2G;
        const bool row_ok = lane < NR && it < Ls;
        int lo = kNoLo, hi = kNoHi;
        if (row_ok) {
            const int pos = c + it;
            lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
            if (p.key_start) lo = max(lo, p.key_start[q0 + it]);
            hi = pos;
            if (p.prefix_lens) hi = max(hi, min(p.prefix_lens[s], n) - 1);
            if (lo > hi) lo = kNoLo, hi = kNoHi;
        }
        if (lane < NR) {
            m_lo[lane] = lo;
            m_hi[lane] = hi;
            m_pos[lane] = (float)it;
            m_slope[lane] = BIAS && row_ok ? p.slopes[g * p.G + (lane & (p.G - 1))] * kLog2e : 0.f;
            m_scale[lane] = p.sl;
            m_nm[lane] = row_ok ? -kNoMax : kNoMax;            // rows there are not: probability 0
        }
        const int a = __reduce_min_sync(~0u, lo), b = __reduce_max_sync(~0u, hi);
        const int d = __reduce_max_sync(~0u, row_ok ? lo : -1);
        const int e = __reduce_min_sync(~0u, row_ok ? hi : INT_MAX);
        if (lane == 0) {
            ranges[0] = a;
            ranges[1] = b;
            ranges[2] = d;
            ranges[3] = e;
            mbar_init(q_full, 1);
            mbar_init(q_ready, NR);
#pragma unroll 1
            for (int i = 0; i < NS; ++i) {
                mbar_init(full(i), FP8 ? 4 : 1);
                mbar_init(free_(i), 1);
            }
#pragma unroll 1
            for (int i = 0; i < RS; ++i) {
                mbar_init(raw_full(i), 1);
                mbar_init(raw_free(i), 4);
            }
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                mbar_init(k_full(i), 4);
                mbar_init(k_free(i), 1);
                mbar_init(s_full(i), 1);
                mbar_init(s_free(i), 4 * NG);
                mbar_init(p_full(i), 4 * NG);
                mbar_init(pv_done(i), 1);
                mbar_init(sync(i), 4);
                flags[i] = flags[2 + i] = 0;
            }
            mbar_init(drain, 2);
            misc[1] = 0;
            dirty[0] = INT_MAX;
            dirty[1] = -1;
            fence_mbar_init();
        }
    } else if (warp == W0 + 1) {
        tmem_alloc(sb + L::MISC, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::MISC);
    auto tS = [&](int b) { return tmem + 32u + 32u * b; };
    auto tK = [&](int b) { return tmem + 128u + 64u * b; };

    // the key tiles of this CTA, as in the kernel for many rows
    const int lo_c = ranges[0], hi_c = ranges[1], maxlo_c = ranges[2], minhi_c = ranges[3];
    const int kbase = hi_c < 0 ? 0 : lo_c & ~(p.bs - 1);
    const int all = hi_c < 0 ? 0 : (hi_c - kbase) / kBN + 1;
    const int parts = p.max_parts == 1 ? 1 : max(1, min(p.max_parts, (all + p.part_tiles - 1) / p.part_tiles));
    const int t0 = parts == 1 ? 0 : part * p.part_tiles;
    const int nt = part >= parts ? 0 : part == parts - 1 ? all - t0 : p.part_tiles;
    const int kb = kbase + t0 * kBN;
    auto masked = [&](int j) { return kb + j * kBN < maxlo_c || kb + j * kBN + kBN - 1 > minhi_c; };
    const int rows = Ls << p.log2G;                            // NR at most
    auto out_row = [&](int r) {
        return (size_t)(q0 + (r >> p.log2G)) * p.Hq + g * p.G + (r & (p.G - 1));
    };

    if (nt == 0) {                                             // CTA-uniform: no key for any row
        if (parts == 1 && part == 0)
#pragma unroll 1
            for (int i = threadIdx.x; i < rows * (D / 8); i += L::THREADS)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + out_row(i / (D / 8)) * (D * 2) + (i % (D / 8)) * 16) =
                    make_uint4(0, 0, 0, 0);
        if (p.max_parts > 1 && (int)threadIdx.x < rows)
            p.ws_ml[out_row(threadIdx.x) * p.max_parts + part] =
                make_float2(-INFINITY, parts == 1 && part == 0 ? -1.f : 0.f);
    } else if (warp == W0) {
        // ------------------------------------------------------------ copies
        const int bpt = kBN >> p.log2bs;                       // blocks per key tile
        const int tpf = 32 / bpt;                              // tiles per 32 table entries
        const uint32_t box = (uint32_t)p.bs * 128u;
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, NSEG * NR * 128);
#pragma unroll 1
            for (int sg = 0; sg < NSEG; ++sg)
                tma_load_3d(sb + L::Q + sg * NR * 128, &tmq, q_full, sg * 64, g * p.G, q0);
        }
        constexpr uint32_t TX = FP8 ? kSeg : L::TILE;
        // 32 table entries a time, the next ones on the way; a block past the last
        // visible key, or an id outside the cache, reads block NB: zeros
        auto entry = [&](int t) {
            const int lb = ((kb + t * kBN) >> p.log2bs) + lane;
            return ((long long)lb << p.log2bs) <= hi_c ? p.block_tables[(size_t)s * p.MB + lb] : INT_MIN;
        };
        // K_j and V_j: the use and the slot of the ring (8-bit: uses 2j, 2j + 1 of one ring)
        auto use = [&](int j, int kv) { return FP8 ? 2 * j + kv : j; };
        auto ring = [&](int kv) { return FP8 ? RS : kv ? VS : KS; };
        auto filled = [&](int kv, int st) { return FP8 ? raw_full(st) : full(kv ? KS + st : st); };
        int started[2] = {0, 0}, next = entry(0), ids = 0;
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j < nt && ok; ++j) {
            if (j % tpf == 0) {
                const int e = next;
                const bool in = e >= 0 && (long long)e < p.NB;
                // entries past this part's last tile are the next part's to judge
                if (!in && e != INT_MIN && j * bpt + lane < nt * bpt) atomicOr(p.err, PA_DEV_BAD_BLOCK);
                ids = in ? e : (int)p.NB;
                next = entry(j + tpf);
            }
            const int id = __shfl_sync(~0u, ids, ((j % tpf) * bpt + lane) & 31);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int u = use(j, kv), st = u % ring(kv), slot = FP8 ? st : kv ? KS + st : st;
                const uint32_t fb = filled(kv, st);
                ok = ok && quick_wait(FP8 ? raw_free(st) : free_(slot), ((u / ring(kv)) & 1) ^ 1, abort_flag,
                                      p.err, 10 + kv);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(fb, TX);
                __syncwarp();
                if (lane < bpt) {
                    if constexpr (FP8) {
                        tma_load_4d_plain(sb + L::RAW + st * kSeg + lane * box, kv ? &tmv : &tmk, fb, 0,
                                          g, 0, id);
                    } else {
#pragma unroll 1
                        for (int sg = 0; sg < NSEG; ++sg)
                            tma_load_4d_plain(sb + L::OP + slot * L::TILE + sg * kSeg + lane * box,
                                              kv ? &tmv : &tmk, fb, sg * 64, g, 0, id);
                    }
                }
                started[FP8 ? 0 : kv] = u + 1;
            }
        }
        // every copy this warp started has landed before the CTA may exit
#pragma unroll 1
        for (int kv = 0; kv < (FP8 ? 1 : 2); ++kv) {
            const int n_st = kv ? started[1] : started[0], r = ring(kv);
#pragma unroll 1
            for (int i = 0; i < r && i < n_st; ++i) {
                const int last = i + (n_st - 1 - i) / r * r;
                quick_wait(filled(kv, i), (last / r) & 1, abort_flag, p.err, 17, false);
            }
        }
        quick_wait(q_full, 0, abort_flag, p.err, 17, false);
    } else if (warp == W0 + 1) {
        // ---------------------------------------------------- MMAs of S^T
        constexpr uint32_t id_s = idesc_f16(OT == PA_BF16 ? 1 : 0, 0, NR);
        const uint32_t khi = (uint32_t)(sdesc(0, 16) >> 32);
        const uint32_t qlo = ((sb + L::Q) >> 4) | (1u << 16);
        bool ok = quick_wait(QCONV ? q_ready : q_full, 0, abort_flag, p.err, 7);
#pragma unroll 1
        for (int j = 0; j < nt && ok; ++j) {
            // K_j: 8-bit in tensor memory, 16-bit in its ring
            constexpr int KR = FP8 ? 1 : KS;
            const int b = j & 1, sk = FP8 ? 0 : j % KR;
            ok = FP8 ? quick_wait(k_full(b), (j >> 1) & 1, abort_flag, p.err, 8)
                     : quick_wait(full(sk), (uint32_t)(j / KR) & 1u, abort_flag, p.err, 8);
            if (ok && j >= 2) ok = quick_wait(s_free(b), ((j >> 1) - 1) & 1, abort_flag, p.err, 12);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
                const uint32_t klo = ((sb + L::OP + sk * L::TILE) >> 4) | (1u << 16);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t qoff = ((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4;
                    if constexpr (FP8)
                        tc_mma_ts_lh(tS(b), tK(b) + kk * 8, qlo + qoff, khi, id_s, kk > 0);
                    else
                        tc_mma_lh(tS(b), klo + (((kk >> 2) * kSeg + (kk & 3) * 32) >> 4), khi, qlo + qoff,
                                  khi, id_s, kk > 0);
                }
                tc_commit(s_full(b));
                tc_commit(FP8 ? k_free(b) : free_(sk));
            }
            __syncwarp();
        }
        // every MMA this warp issued completes before tensor memory is freed
        if (lane == 0) tc_commit(drain);
        __syncwarp();
        quick_wait(drain, 0, abort_flag, p.err, 16, false);
    } else if (warp == W0 + 2) {
        // ------------------- MMAs of O^T, and 16-bit the look through V
        // both operands MN-major (bit 15: A, V^T, too)
        constexpr uint32_t id_o = idesc_f16(OT == PA_BF16 ? 1 : 0, 1, NR) | (1u << 15);
        const uint32_t mhi = (uint32_t)(sdesc(0, kSeg) >> 32);
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
            const int b = j & 1, sv = KS + j % VS;
            if (!(ok = quick_wait(full(sv), (uint32_t)(j / VS) & 1u, abort_flag, p.err, 9))) break;
            if (!FP8 && masked(j)) {
                const uint32_t tile = sb + L::OP + sv * L::TILE + lane * 16;
                bool bad = false;
#pragma unroll 8
                for (int v = 0; v < L::TILE; v += 512) bad |= nonfinite<OT>(lds128(tile + v));
                if (__any_sync(~0u, bad)) {
#pragma unroll 1
                    for (int v = 0; v < L::TILE; v += 512) sts128(tile + v, finite_only<OT>(lds128(tile + v)));
                    if (lane == 0) {
                        atomicMin(dirty, j);
                        atomicMax(dirty + 1, j);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (!(ok = quick_wait(p_full(b), (j >> 1) & 1, abort_flag, p.err, 13))) break;
            tc_fence_after();
            if (lane == 0) {
                // D = 64: rows 64..127 of the product are of no use (their operand
                // is whatever lies behind the tile)
                const uint32_t vlo = ((sb + L::OP + sv * L::TILE) >> 4) | ((uint32_t)(kSeg >> 4) << 16);
                const uint32_t plo = ((sb + L::P + b * kSeg) >> 4) | ((uint32_t)(kSeg >> 4) << 16);
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    tc_mma_lh(tmem, vlo + kk * 128, mhi, plo + kk * 128, mhi, id_o, (j > 0 || kk > 0) ? 1u : 0u);
                tc_commit(pv_done(b));
                tc_commit(free_(sv));
            }
            __syncwarp();
        }
        if (lane == 0) tc_commit(drain);
        __syncwarp();
        quick_wait(drain, 0, abort_flag, p.err, 16, false);
    } else if (warp >= W0 + 4) {
        // ------------------------------------------- E4M3 codes to f16 operands
        if constexpr (FP8) {
            const int tid = threadIdx.x - 32 * (W0 + 4);       // K: this thread's key
            const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
#pragma unroll 1
            for (int j = 0; j < nt; ++j) {
                {
                    const int u = 2 * j, rs = u % RS, b = j & 1;
                    if (!quick_wait(raw_full(rs), (u / RS) & 1, abort_flag, p.err, 9)) break;
                    const uint32_t src = sb + L::RAW + rs * kSeg;
                    uint4 w[8];
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) w[ch] = lds128(src + swz128(tid, ch));
                    if (j >= 2 && !quick_wait(k_free(b), ((j >> 1) - 1) & 1, abort_flag, p.err, 10)) break;
                    tc_fence_after();
#pragma unroll
                    for (int c2 = 0; c2 < 4; ++c2) {
                        uint32_t h[16];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint4 v = w[2 * c2 + e];
                            const uint2 a = widen(v.x), bb = widen(v.y), cc = widen(v.z), d = widen(v.w);
                            h[8 * e + 0] = a.x, h[8 * e + 1] = a.y, h[8 * e + 2] = bb.x, h[8 * e + 3] = bb.y;
                            h[8 * e + 4] = cc.x, h[8 * e + 5] = cc.y, h[8 * e + 6] = d.x, h[8 * e + 7] = d.y;
                        }
                        tmem_st16(tK(b) + lrow + c2 * 16, h);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(k_full(b));
                        mbar_arrive(raw_free(rs));
                    }
                }
                const int u = 2 * j + 1, rs = u % RS, st = j % VS;
                if (!quick_wait(raw_full(rs), (u / RS) & 1, abort_flag, p.err, 9)) break;
                const uint32_t src = sb + L::RAW + rs * kSeg;
                const uint32_t dst = sb + L::OP + st * L::TILE;
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = lds128(src + swz128((tid >> 3) + 16 * i, tid & 7));
                if (j >= VS && !quick_wait(free_(st), (uint32_t)(j / VS - 1) & 1u, abort_flag, p.err, 10)) break;
                const bool look = masked(j);
                bool bad = false;
                const int ch = tid & 7, oc = 2 * (ch & 3), sw = ch >> 2;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // as in the kernel for many rows: chunk ch of row t
                    const int t = (tid >> 3) + 16 * i;
                    const uint2 h0 = widen(w[i].x), h1 = widen(w[i].y), h2 = widen(w[i].z), h3 = widen(w[i].w);
                    const uint4 a = make_uint4(h0.x, h0.y, h1.x, h1.y), b = make_uint4(h2.x, h2.y, h3.x, h3.y);
                    if (look) bad |= nonfinite<PA_F16>(a) | nonfinite<PA_F16>(b);
                    const uint32_t seg = dst + sw * kSeg;
                    sts128(seg + swz128(t, oc + sw), sw ? b : a);
                    sts128(seg + swz128(t, oc + 1 - sw), sw ? a : b);
                }
                if (bad) {                                    // this thread's chunks once more
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t at = dst + sw * kSeg + swz128((tid >> 3) + 16 * (i >> 1), oc + (i & 1));
                        sts128(at, finite_only<PA_F16>(lds128(at)));
                    }
                    atomicMin(dirty, j);
                    atomicMax(dirty + 1, j);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full(st));
                    mbar_arrive(raw_free(rs));
                }
            }
        }
    } else if (warp < W0) {
        // ---------- softmax: this thread's key of every tile, 16 of the rows
        constexpr int R = 16;
        const int q = warp >> 2, r0 = q * R, t = threadIdx.x & 127;
        const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
        float* xch = reinterpret_cast<float*>(sm + L::XCH + r0 * L::XROW);
        constexpr int XF = L::XROW / 4;
        bool ok = true;
        uint32_t nsync = 0;
        // the group's four warps; bounded like every other wait
        auto arrive = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(sync(q));
        };
        auto joined = [&]() { return quick_wait(sync(q), nsync++ & 1, abort_flag, p.err, 21); };
        if constexpr (QCONV) {
            ok = quick_wait(q_full, 0, abort_flag, p.err, 7);
            if (ok && t < R) {
                m_scale[r0 + t] = p.sl * row_to_f16<D, NR * 128>(sb + L::Q, r0 + t);
                fence_proxy_async_smem();
                mbar_arrive(q_ready);
            }
            arrive();
            ok = ok && joined();
        }
        // SHIFT - the rows' references, this key's part of their sums, their factors
        float nm[R], l[R], sc[QCONV ? R : 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            nm[r] = m_nm[r0 + r];
            l[r] = 0.f;
            if constexpr (QCONV) sc[r] = m_scale[r0 + r];
        }
#pragma unroll 1
        for (int j = 0; j < nt && ok; ++j) {
            const int b = j & 1;
            if (!(ok = quick_wait(s_full(b), (j >> 1) & 1, abort_flag, p.err, 12))) break;
            tc_fence_after();
            float z[R];
            tmem_ld16(tS(b) + lrow + r0, z);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free(b));
            const int key = kb + j * kBN + t;
            // scores in log2 units
            float most[4] = {};
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                const float2 u = mul2(make_float2(z[r], z[r + 1]),
                                      QCONV ? make_float2(sc[r], sc[r + 1]) : make_float2(p.sl, p.sl));
                z[r] = u.x;
                z[r + 1] = u.y;
                if constexpr (CAP) most[(r >> 1) & 3] = max3(most[(r >> 1) & 3], fabsf(u.x), fabsf(u.y));
            }
            if constexpr (CAP) {
                const float cl = p.cap_log2;
                float2 co[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) co[k] = make_float2(kTanh4[k] * cl, kTanh4[k] * cl);
                // |u| <= 2: the four-term fit; beyond, the special-function unit.  What a score
                // becomes depends on its own size alone; the vote only saves the second form.
                auto capped = [&](auto far) {
#pragma unroll
                    for (int r = 0; r < R; r += 2) {
                        const float2 u = make_float2(z[r], z[r + 1]), v = mul2(u, u);
                        const float2 y = mul2(u, fma2(fma2(fma2(co[3], v, co[2]), v, co[1]), v, co[0]));
                        z[r] = decltype(far)::value && !(fabsf(u.x) <= 2.f) ? cl * tanh_quarter(u.x) : y.x;
                        z[r + 1] = decltype(far)::value && !(fabsf(u.y) <= 2.f) ? cl * tanh_quarter(u.y) : y.y;
                    }
                };
                if (__any_sync(~0u, fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) > 2.f)) capped(std::true_type());
                else capped(std::false_type());
            }
            if constexpr (BIAS) {
                // positions counted from the first new token: a distance between numbers that
                // fp32 holds exactly (past 2^24 it does not hold positions)
                const float kf = (float)(key - c);
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 at = *reinterpret_cast<const float4*>(m_pos + r0 + r);
                    const float4 sp = *reinterpret_cast<const float4*>(m_slope + r0 + r);
                    z[r] = fmaf(-sp.x, fabsf(at.x - kf), z[r]);
                    z[r + 1] = fmaf(-sp.y, fabsf(at.y - kf), z[r + 1]);
                    z[r + 2] = fmaf(-sp.z, fabsf(at.z - kf), z[r + 2]);
                    z[r + 3] = fmaf(-sp.w, fabsf(at.w - kf), z[r + 3]);
                }
            }
            if (masked(j)) {
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const int4 lo = *reinterpret_cast<const int4*>(m_lo + r0 + r);
                    const int4 hi = *reinterpret_cast<const int4*>(m_hi + r0 + r);
                    if (key < lo.x || key > hi.x) z[r] = -INFINITY;
                    if (key < lo.y || key > hi.y) z[r + 1] = -INFINITY;
                    if (key < lo.z || key > hi.z) z[r + 2] = -INFINITY;
                    if (key < lo.w || key > hi.w) z[r + 3] = -INFINITY;
                }
            }
            // does a score exceed its row's reference by more than 8?
            float pr[R], top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                const float2 d = add2(make_float2(z[r], z[r + 1]), make_float2(nm[r], nm[r + 1]));
                pr[r] = d.x;
                pr[r + 1] = d.y;
                top[(r >> 1) & 3] = max3(top[(r >> 1) & 3], d.x, d.y);
            }
            const float over = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            if (__any_sync(~0u, over > kRescaleLog2 + SHIFT) && lane == 0) flags[2 * q + b] = j + 1;
            arrive();
            // the probabilities, in case no warp found one (the wait is over by then)
#pragma unroll
            for (int r = 0; r < R; ++r) pr[r] = ex2(pr[r]);
            if (!(ok = joined())) break;
            if (flags[2 * q + b] == j + 1) {
                // the tile's maxima, and everything so far against them
#pragma unroll
                for (int r = 0; r < R; ++r) xch[r * XF + t] = z[r];
                arrive();
                if (!(ok = joined())) break;
#pragma unroll 1
                for (int r = warp & 3; r < R; r += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(xch + r * XF + lane * 4);
                    const float fresh = SHIFT - warp_max(max3(v.x, v.y, fmaxf(v.z, v.w)));
                    if (lane == 0) {
                        // The reference of a row that sees nothing, or is not there, stays, and
                        // that of a row that did not ask: what another row sees is not to
                        // change a bit of it.
                        const float old = m_nm[r0 + r];
                        const bool raise = r0 + r < rows && old - fresh > kRescaleLog2;
                        m_alpha[r0 + r] = raise ? ex2(fresh - old) : 1.f;
                        if (raise) m_nm[r0 + r] = fresh;
                    }
                }
                // O^T holds the tiles before once the last of them completes
                if (j > 0 && !(ok = quick_wait(pv_done(b ^ 1), ((j - 1) >> 1) & 1, abort_flag, p.err, 14))) break;
                arrive();
                if (!(ok = joined())) break;
                tc_fence_after();
                float o[R];
                tmem_ld16(tmem + lrow + r0, o);                // (the first tile's: of no use)
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = m_alpha[r0 + r];
                    nm[r] = m_nm[r0 + r];
                    l[r] *= f;
                    o[r] *= f;
                    pr[r] = ex2(z[r] + nm[r]);
                }
                tmem_st16(tmem + lrow + r0, reinterpret_cast<const uint32_t*>(o));
                tmem_wait_st();
            }
            uint32_t w[R / 2];
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                const float2 a = add2(make_float2(l[r], l[r + 1]), make_float2(pr[r], pr[r + 1]));
                l[r] = a.x;
                l[r + 1] = a.y;
                w[r / 2] = pack2<OT>(pr[r], pr[r + 1]);
            }
            if (j >= 2 && !(ok = quick_wait(pv_done(b), ((j >> 1) - 1) & 1, abort_flag, p.err, 14))) break;
            const uint32_t row = sb + L::P + b * kSeg;
            sts128(row + swz128(t, 2 * q), make_uint4(w[0], w[1], w[2], w[3]));
            sts128(row + swz128(t, 2 * q + 1), make_uint4(w[4], w[5], w[6], w[7]));
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(b));
        }
        // -------------------------------------------------------- epilogue
        if (p.max_parts > 1) launch_dependents();              // the join may start launching
        const bool record = parts > 1;
        const int mine = min(rows - r0, R);                    // rows of this group (or none)
        if (ok) ok = quick_wait(pv_done((nt - 1) & 1), ((nt - 1) >> 1) & 1, abort_flag, p.err, 15);
        tc_fence_after();
        // sums and outputs change hands through the exchange rows
#pragma unroll
        for (int r = 0; r < R; ++r) xch[r * XF + t] = l[r];
        arrive();
        if (ok) ok = joined();
        if (ok) {
#pragma unroll 1
            for (int r = warp & 3; r < mine; r += 4) {
                const float4 v = *reinterpret_cast<const float4*>(xch + r * XF + lane * 4);
                float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                if (lane == 0) {
                    m_sum[r0 + r] = sum;
                    // l = -1 marks a row that needs no join
                    if (p.max_parts > 1)
                        p.ws_ml[out_row(r0 + r) * p.max_parts + part] =
                            make_float2(SHIFT - m_nm[r0 + r], record ? sum : -1.f);
                }
            }
        }
        arrive();
        if (ok) ok = joined();
        if (ok && (warp & 3) * 32 < D) {
            float o[R];
            tmem_ld16(tmem + lrow + r0, o);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < R; ++r) xch[r * XF + t] = o[r];
            if (dirty[1] >= 0) {                               // values were taken out of V
                const int ka = max(lo_c, kb + dirty[0] * kBN);
                const int kz = min(hi_c, kb + dirty[1] * kBN + kBN - 1);
#pragma unroll 1
                for (int k = ka; k <= kz; ++k) {
                    if (!masked((k - kb) >> 7)) {              // this tile kept its values
                        k = kb + ((k - kb) | (kBN - 1));
                        continue;
                    }
                    const int id = p.block_tables[(size_t)s * p.MB + (k >> p.log2bs)];
                    if (id < 0 || (long long)id >= p.NB) continue;
                    const float y = cache_value<FP8 ? (int)PA_FP8_E4M3 : QT>(
                        p.v_cache, (((size_t)id * p.bs + (k & (p.bs - 1))) * heads + g) * D + t);
                    if (isfinite(y)) continue;
#pragma unroll 1
                    for (int r = 0; r < mine; ++r)
                        if (k >= m_lo[r0 + r] && k <= m_hi[r0 + r]) xch[r * XF + t] += y;
                }
            }
        }
        arrive();
        if (ok) ok = joined();
        if (ok) {
            // 8 dims of a row a thread
#pragma unroll 1
            for (int i = t; i < mine * (D / 8); i += 128) {
                const int r = i / (D / 8), d = i % (D / 8) * 8;
                const float4* src = reinterpret_cast<const float4*>(xch + r * XF + d);
                const float4 a = src[0], b = src[1];
                if (record) {
                    float4* dst = reinterpret_cast<float4*>(p.ws_o + (out_row(r0 + r) * p.max_parts + part) * D + d);
                    dst[0] = a;
                    dst[1] = b;
                } else {
                    const float sum = m_sum[r0 + r], f = sum == 0.f ? 0.f : p.v_scale / sum;
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (out_row(r0 + r) * D + d) * 2) =
                        make_uint4(pack2<QT>(a.x * f, a.y * f), pack2<QT>(a.z * f, a.w * f),
                                   pack2<QT>(b.x * f, b.y * f), pack2<QT>(b.z * f, b.w * f));
                }
            }
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == W0 + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int QT, bool FP8, int D, int NR, bool CAP, bool BIAS>
cudaError_t launch_few_one(const Launch& a) {
    using L = FewPlan<FP8, D, NR>;
    const cudaError_t e = ensure_dynamic_smem<prefill_few_kernel<QT, FP8, D, NR, CAP, BIAS>>(L::BYTES);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefill_few_kernel<QT, FP8, D, NR, CAP, BIAS>, a.grid, dim3(L::THREADS),
                      (size_t)L::BYTES, a.stream, *a.mq, *a.mk, *a.mv, *a.p);
}

template <int QT, bool FP8, int D>
cudaError_t launch_few(const Launch& a) {
    const bool cap = a.p->cap_log2 > 0.f, bias = a.p->slopes != nullptr;
    auto by_mod = [&](auto nr) {
        constexpr int NR = decltype(nr)::value;
        if (cap) return bias ? launch_few_one<QT, FP8, D, NR, true, true>(a) : launch_few_one<QT, FP8, D, NR, true, false>(a);
        return bias ? launch_few_one<QT, FP8, D, NR, false, true>(a) : launch_few_one<QT, FP8, D, NR, false, false>(a);
    };
    const cudaError_t e = a.few == 16 ? by_mod(std::integral_constant<int, 16>()) : by_mod(std::integral_constant<int, 32>());
    return e == cudaSuccess ? launch_merge<QT, D>(a) : e;
}

}  // namespace ps
