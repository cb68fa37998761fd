// Chunk attention with modified scores for few query rows (pa_prefill_scored,
// at most 32 rows of a kv head: L new tokens x G query heads), bound by the read
// of the cache.
//
// With few rows the roles of keys and queries are exchanged, so that the 128 rows
// of the MMA are keys and the few queries its columns:
//     S_j^T = K_j Q^T    128 keys x NR rows, one key per softmax thread
//     O^T  += V_j^T P_j^T   D x NR, V the MN-major A operand, P written to shared
//                        memory in the layout of V
// A softmax thread has NR scores instead of 128, four warps share the
// exponentials of a tile, and the next scores are computed meanwhile (S_j^T takes
// NR columns, so two fit).  The price is that a row's maximum lies across
// threads.  It is not needed every tile: scores are taken against the running
// reference m of their row, and only when one exceeds it by more than 8 (in log2
// units; the first tile always) the four warps find the tile's maxima (a warp
// reduction a row) and rescale.  A row's sum is kept per thread and added up once.
//
// 8-bit cache: four more warps widen the codes to f16 (exactly): K to tensor
// memory, from where the MMA takes it as its A operand, so it does not pass
// through shared memory again; V to shared memory.  Per 128-key tile of D = 128
// shared memory then moves 256 cycles' worth of arriving codes, 256 read back, 256
// of V written and 256 read by the MMA, and P; HBM brings the tile's 32 KB in
// 1400 cycles an SM.  A bf16 query row is scaled as in the kernel for many rows.
//
// Warps: 0-3 softmax, epilogue; 4 copies; 5 MMAs; 6, 7 idle; 8-bit: 8-11 widening.
// Tensor memory: O^T from 0, S^T from 32 and 64, K operands from 128 and 192.
// Waits are bounded and non-finite values handled as in the kernel for many rows.
#pragma once

#include "prefill_scored.cuh"

namespace ps {

template <bool FP8, int D, int NR>
struct FewPlan {
    static constexpr int NSEG = D / 64;
    static constexpr int TILE = NSEG * kSeg;
    // 16-bit: ring of K and V tiles in turn; 8-bit: two V operand tiles, ring of codes
    static constexpr int NS = FP8 ? 2 : D == 64 ? 10 : 5;
    static constexpr int RS = FP8 ? 7 : 0;
    static constexpr int QB = NR * 128 * NSEG;
    static constexpr int Q = 0;
    static constexpr int OP = QB;
    static constexpr int RAW = OP + NS * TILE;
    static constexpr int P = RAW + RS * kSeg;           // 2 x 128 keys x 128 bytes
    static constexpr int META = P + 2 * kSeg;
    // rows: lo, hi, position, slope, factor of their scores, alpha, 1 / sum; part[4][NR]
    static constexpr int METAB = NR * 4 * (7 + 4);
    static constexpr int BAR = META + METAB;
    // q_full, q_ready, full[NS], free[NS], raw_full[RS], raw_free[RS], k_full[2],
    // k_free[2], s_full[2], s_free[2], p_full[2], pv_done[2], sync, drain
    static constexpr int NBAR = 2 + 2 * NS + 2 * RS + 12 + 2;
    static constexpr int MISC = BAR + NBAR * 8;         // tensor memory, abort, dirty, flags, ranges
    static constexpr int BYTES = MISC + 64 + 1024;
    static_assert(BYTES <= 232448, "shared memory of one CTA");
    static constexpr int THREADS = FP8 ? 384 : 256;
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
    constexpr int NSEG = L::NSEG, NS = L::NS, RS = L::RS;
    constexpr bool QCONV = FP8 && QT == PA_BF16;
    constexpr float SHIFT = OT == PA_F16 ? 7.f : 0.f;      // as in the kernel for many rows
    grid_dependency_wait();
    const int part = (int)blockIdx.x % p.max_parts, g = (int)blockIdx.x / p.max_parts;
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
    const uint32_t sync = bx + 96u, drain = bx + 104u;
    volatile int* misc = reinterpret_cast<volatile int*>(sm + L::MISC);
    volatile int* abort_flag = misc + 1;
    int* dirty = reinterpret_cast<int*>(sm + L::MISC) + 2;     // first, last tile with zeroed values
    volatile int* flags = misc + 4;                            // 2: tile + 1 whose maximum was raised
    int* ranges = reinterpret_cast<int*>(sm + L::MISC) + 6;    // lo, hi, largest lo, smallest hi
    int* m_lo = reinterpret_cast<int*>(sm + L::META);
    int* m_hi = m_lo + NR;
    float* m_pos = reinterpret_cast<float*>(m_lo + 2 * NR);
    float* m_slope = m_pos + NR;
    float* m_scale = m_pos + 2 * NR;
    float* m_alpha = m_pos + 3 * NR;
    float* m_inv = m_pos + 4 * NR;
    float* m_part = m_pos + 5 * NR;                            // [4][NR]

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
            m_pos[lane] = (float)(c + it);
            m_slope[lane] = BIAS && row_ok ? p.slopes[g * p.G + (lane & (p.G - 1))] * kLog2e : 0.f;
            m_scale[lane] = p.sl;
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
            for (int i = 0; i < NS; ++i) {
                mbar_init(full(i), FP8 ? 4 : 1);
                mbar_init(free_(i), 1);
            }
            for (int i = 0; i < RS; ++i) {
                mbar_init(raw_full(i), 1);
                mbar_init(raw_free(i), 4);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(k_full(i), 4);
                mbar_init(k_free(i), 1);
                mbar_init(s_full(i), 1);
                mbar_init(s_free(i), 4);
                mbar_init(p_full(i), 4);
                mbar_init(pv_done(i), 1);
                flags[i] = 0;
            }
            mbar_init(sync, 4);
            mbar_init(drain, 1);
            misc[1] = 0;
            dirty[0] = INT_MAX;
            dirty[1] = -1;
            fence_mbar_init();
        }
    } else if (warp == 5) {
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
            for (int i = threadIdx.x; i < rows * (D / 8); i += L::THREADS)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + out_row(i / (D / 8)) * (D * 2) + (i % (D / 8)) * 16) =
                    make_uint4(0, 0, 0, 0);
        if (p.max_parts > 1 && (int)threadIdx.x < rows)
            p.ws_ml[out_row(threadIdx.x) * p.max_parts + part] =
                make_float2(-INFINITY, parts == 1 && part == 0 ? -1.f : 0.f);
    } else if (warp == 4) {
        // ------------------------------------------------------------ copies
        const int bpt = kBN >> p.log2bs;                       // blocks per key tile
        const int tpf = 32 / bpt;                              // tiles per 32 table entries
        const uint32_t box = (uint32_t)p.bs * 128u;
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, NSEG * NR * 128);
            for (int sg = 0; sg < NSEG; ++sg)
                tma_load_3d(sb + L::Q + sg * NR * 128, &tmq, q_full, sg * 64, g * p.G, q0);
        }
        constexpr int RING = FP8 ? RS : NS;
        constexpr uint32_t TX = FP8 ? kSeg : L::TILE;
        // 32 table entries a time, the next ones on the way; a block past the last
        // visible key, or an id outside the cache, reads block NB: zeros
        auto entry = [&](int t) {
            const int lb = ((kb + t * kBN) >> p.log2bs) + lane;
            return ((long long)lb << p.log2bs) <= hi_c ? p.block_tables[(size_t)s * p.MB + lb] : INT_MIN;
        };
        int started = 0, next = entry(0), ids = 0;
        for (int j = 0; j < nt; ++j) {
            if (j % tpf == 0) {
                const int e = next;
                const bool in = e >= 0 && (long long)e < p.NB;
                // entries past this part's last tile are the next part's to judge
                if (!in && e != INT_MIN && j * bpt + lane < nt * bpt) atomicOr(p.err, PA_DEV_BAD_BLOCK);
                ids = in ? e : (int)p.NB;
                next = entry(j + tpf);
            }
            const int id = __shfl_sync(~0u, ids, ((j % tpf) * bpt + lane) & 31);
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
                        tma_load_4d_plain(sb + L::RAW + st * kSeg + lane * box, kv ? &tmv : &tmk, fb, 0,
                                          g, 0, id);
                    } else {
                        for (int sg = 0; sg < NSEG; ++sg)
                            tma_load_4d_plain(sb + L::OP + st * L::TILE + sg * kSeg + lane * box,
                                              kv ? &tmv : &tmk, fb, sg * 64, g, 0, id);
                    }
                }
                started = u + 1;
            }
            if (!ok) break;
        }
        // every copy this warp started has landed before the CTA may exit
        for (int i = 0; i < RING && i < started; ++i) {
            const int last = i + (started - 1 - i) / RING * RING;
            warp_wait(FP8 ? raw_full(i) : full(i), (last / RING) & 1, abort_flag, p.err, 17, false);
        }
        warp_wait(q_full, 0, abort_flag, p.err, 17, false);
    } else if (warp == 5) {
        // -------------------------------------------------------------- MMAs
        constexpr int ABF = OT == PA_BF16 ? 1 : 0;
        const uint32_t id_s = idesc_f16(ABF, 0, NR);
        const uint32_t id_o = idesc_f16(ABF, 1, NR) | (1u << 15);       // A (V^T) MN-major too
        const uint32_t khi = (uint32_t)(sdesc(0, 16) >> 32), mhi = (uint32_t)(sdesc(0, kSeg) >> 32);
        const uint32_t qlo = ((sb + L::Q) >> 4) | (1u << 16);
        // K_j, V_j: 16-bit slots 2j, 2j + 1 of the ring; 8-bit tensor memory, slot j
        auto kslot = [&](int j) { return FP8 ? 0 : (2 * j) % NS; };
        auto vslot = [&](int j) { return FP8 ? j % NS : (2 * j + 1) % NS; };
        auto vphase = [&](int j) { return (uint32_t)((FP8 ? j : 2 * j + 1) / NS) & 1u; };
        auto issue_s = [&](int j) {
            const int b = j & 1;
            if (FP8) {
                if (!warp_wait(k_full(b), (j >> 1) & 1, abort_flag, p.err, 8)) return false;
            } else {
                if (!warp_wait(full(kslot(j)), (uint32_t)(2 * j / NS) & 1u, abort_flag, p.err, 8)) return false;
            }
            if (j >= 2 && !warp_wait(s_free(b), ((j >> 1) - 1) & 1, abort_flag, p.err, 12)) return false;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t qoff = ((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4;
                    if constexpr (FP8) {
                        tc_mma_ts_lh(tS(b), tK(b) + kk * 8, qlo + qoff, khi, id_s, kk > 0);
                    } else {
                        const uint32_t klo = ((sb + L::OP + kslot(j) * L::TILE) >> 4) | (1u << 16);
                        tc_mma_lh(tS(b), klo + (((kk >> 2) * kSeg + (kk & 3) * 32) >> 4), khi, qlo + qoff,
                                  khi, id_s, kk > 0);
                    }
                }
                tc_commit(s_full(b));
                tc_commit(FP8 ? k_free(b) : free_(kslot(j)));
            }
            __syncwarp();
            return true;
        };
        bool ok = warp_wait(QCONV ? q_ready : q_full, 0, abort_flag, p.err, 7) && issue_s(0);
        for (int j = 0; j < nt && ok; ++j) {
            if (j + 1 < nt && !(ok = issue_s(j + 1))) break;
            const int b = j & 1, sv = vslot(j);
            if (!(ok = warp_wait(full(sv), vphase(j), abort_flag, p.err, 9))) break;
            if (!FP8 && masked(j)) {
                uint4* tile = reinterpret_cast<uint4*>(sm + L::OP + sv * L::TILE);
                bool bad = false;
#pragma unroll 8
                for (int v = lane; v < L::TILE / 16; v += 32) bad |= nonfinite<OT>(tile[v]);
                if (__any_sync(~0u, bad)) {
                    for (int v = lane; v < L::TILE / 16; v += 32) tile[v] = finite_only<OT>(tile[v]);
                    if (lane == 0) {
                        atomicMin(dirty, j);
                        atomicMax(dirty + 1, j);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
            if (!(ok = warp_wait(p_full(b), (j >> 1) & 1, abort_flag, p.err, 13))) break;
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
        // every MMA this warp issued completes before tensor memory is freed
        if (lane == 0) tc_commit(drain);
        __syncwarp();
        warp_wait(drain, 0, abort_flag, p.err, 16, false);
    } else if (warp >= 8) {
        // ------------------------------------------- E4M3 codes to f16 operands
        if constexpr (FP8) {
            const int tid = threadIdx.x - 256;                 // K: this thread's key
            const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
            for (int j = 0; j < nt; ++j) {
                {
                    const int u = 2 * j, rs = u % RS, b = j & 1;
                    if (!warp_wait(raw_full(rs), (u / RS) & 1, abort_flag, p.err, 9)) break;
                    const uint8_t* src = sm + L::RAW + rs * kSeg;
                    uint4 w[8];
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) w[ch] = *reinterpret_cast<const uint4*>(src + swz128(tid, ch));
                    if (j >= 2 && !warp_wait(k_free(b), ((j >> 1) - 1) & 1, abort_flag, p.err, 10)) break;
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
                const int u = 2 * j + 1, rs = u % RS, st = j % NS;
                if (!warp_wait(raw_full(rs), (u / RS) & 1, abort_flag, p.err, 9)) break;
                const uint8_t* src = sm + L::RAW + rs * kSeg;
                uint8_t* dst = sm + L::OP + st * L::TILE;
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = *reinterpret_cast<const uint4*>(src + swz128((tid >> 3) + 16 * i, tid & 7));
                if (j >= NS && !warp_wait(free_(st), (uint32_t)(j / NS - 1) & 1u, abort_flag, p.err, 10)) break;
                const bool look = masked(j);
                bool bad = false;
                const int ch = tid & 7, oc = 2 * (ch & 3), sw = ch >> 2;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // as in the kernel for many rows: chunk ch of row t
                    const int t = (tid >> 3) + 16 * i;
                    const uint2 h0 = widen(w[i].x), h1 = widen(w[i].y), h2 = widen(w[i].z), h3 = widen(w[i].w);
                    uint4 a = make_uint4(h0.x, h0.y, h1.x, h1.y), b = make_uint4(h2.x, h2.y, h3.x, h3.y);
                    if (look && (nonfinite<PA_F16>(a) || nonfinite<PA_F16>(b))) {
                        a = finite_only<PA_F16>(a);
                        b = finite_only<PA_F16>(b);
                        bad = true;
                    }
                    uint8_t* seg = dst + sw * kSeg;
                    *reinterpret_cast<uint4*>(seg + swz128(t, oc + sw)) = sw ? b : a;
                    *reinterpret_cast<uint4*>(seg + swz128(t, oc + 1 - sw)) = sw ? a : b;
                }
                if (bad) {
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
    } else if (warp < 4) {
        // ------------------------- softmax: this thread's key of every tile
        const uint32_t lrow = (uint32_t)(warp * 32) << 16;
        bool ok = true;
        uint32_t nsync = 0;
        // all four warps; bounded like every other wait
        auto join = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(sync);
            return warp_wait(sync, nsync++ & 1, abort_flag, p.err, 19);
        };
        if constexpr (QCONV) {
            ok = warp_wait(q_full, 0, abort_flag, p.err, 7);
            if (ok && (int)threadIdx.x < NR) {
                m_scale[threadIdx.x] = p.sl * row_to_f16<D, NR * 128>(sm + L::Q, threadIdx.x);
                fence_proxy_async_smem();
                mbar_arrive(q_ready);
            }
            ok = ok && join();
        }
        float nm[NR], l[NR];                                   // SHIFT - m, and this key's part of the sum
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            nm[r] = r < rows ? -kNoMax : kNoMax;               // rows there are not: probability 0
            l[r] = 0.f;
        }
        for (int j = 0; j < nt && ok; ++j) {
            const int b = j & 1;
            if (!(ok = warp_wait(s_full(b), (j >> 1) & 1, abort_flag, p.err, 12))) break;
            tc_fence_after();
            float z[NR];
            if constexpr (NR == 32) tmem_ld32(tS(b) + lrow, z);
            else tmem_ld16(tS(b) + lrow, z);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free(b));
            const int key = kb + j * kBN + (int)threadIdx.x;
            // scores in log2 units
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                const float4 f = QCONV ? *reinterpret_cast<const float4*>(m_scale + r)
                                       : make_float4(p.sl, p.sl, p.sl, p.sl);
                z[r] *= f.x, z[r + 1] *= f.y, z[r + 2] *= f.z, z[r + 3] *= f.w;
            }
            if constexpr (CAP) {
                const float cl = p.cap_log2;
                float top = 0.f;
#pragma unroll
                for (int r = 0; r < NR; r += 2) top = max3(top, fabsf(z[r]), fabsf(z[r + 1]));
                if (!__any_sync(~0u, !(top <= 4.f))) {
                    float2 co[7];
#pragma unroll
                    for (int t = 0; t < 7; ++t) co[t] = make_float2(kTanh7[t] * cl, kTanh7[t] * cl);
#pragma unroll
                    for (int r = 0; r < NR; r += 2) {
                        const float2 u = make_float2(z[r], z[r + 1]), v = mul2(u, u);
                        float2 y = co[6];
#pragma unroll
                        for (int t = 5; t >= 0; --t) y = fma2(y, v, co[t]);
                        y = mul2(u, y);
                        z[r] = y.x;
                        z[r + 1] = y.y;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < NR; ++r) z[r] = cl * tanh_quarter(z[r]);
                }
            }
            if constexpr (BIAS) {
                const float kf = (float)key;
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 at = *reinterpret_cast<const float4*>(m_pos + r);
                    const float4 sp = *reinterpret_cast<const float4*>(m_slope + r);
                    z[r] = fmaf(-sp.x, fabsf(at.x - kf), z[r]);
                    z[r + 1] = fmaf(-sp.y, fabsf(at.y - kf), z[r + 1]);
                    z[r + 2] = fmaf(-sp.z, fabsf(at.z - kf), z[r + 2]);
                    z[r + 3] = fmaf(-sp.w, fabsf(at.w - kf), z[r + 3]);
                }
            }
            if (masked(j)) {
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const int4 lo = *reinterpret_cast<const int4*>(m_lo + r);
                    const int4 hi = *reinterpret_cast<const int4*>(m_hi + r);
                    if (key < lo.x || key > hi.x) z[r] = -INFINITY;
                    if (key < lo.y || key > hi.y) z[r + 1] = -INFINITY;
                    if (key < lo.z || key > hi.z) z[r + 2] = -INFINITY;
                    if (key < lo.w || key > hi.w) z[r + 3] = -INFINITY;
                }
            }
            // does a score exceed its row's reference by more than 8?
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int r = 0; r < NR; r += 2)
                top[(r >> 1) & 3] = max3(top[(r >> 1) & 3], z[r] + nm[r], z[r + 1] + nm[r + 1]);
            const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            if (__any_sync(~0u, most > kRescaleLog2 + SHIFT) && lane == 0) flags[b] = j + 1;
            if (!(ok = join())) break;
            if (flags[b] == j + 1) {
                // the tile's maxima, and everything so far against them
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float m = warp_max(z[r]);
                    if (lane == 0) m_part[warp * NR + r] = m;
                }
                if (!(ok = join())) break;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float m = fmaxf(fmaxf(m_part[r], m_part[NR + r]),
                                          fmaxf(m_part[2 * NR + r], m_part[3 * NR + r]));
                    const float fresh = SHIFT - m;
                    // nm of a row without a maximum stays; of a row there is not, too
                    float f = 1.f;
                    if (r < rows && fresh < nm[r]) {
                        f = ex2(fresh - nm[r]);
                        nm[r] = fresh;
                    }
                    l[r] *= f;
                    if (threadIdx.x == 0) m_alpha[r] = f;
                }
                if (!(ok = join())) break;
                if (j > 0) {
                    // O^T holds the tiles before once the last of them completes
                    if (!(ok = warp_wait(pv_done(b ^ 1), ((j - 1) >> 1) & 1, abort_flag, p.err, 14))) break;
                    tc_fence_after();
                    float o[NR];
                    if constexpr (NR == 32) tmem_ld32(tmem + lrow, o);
                    else tmem_ld16(tmem + lrow, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < NR; ++r) o[r] *= m_alpha[r];
                    if constexpr (NR == 32) tmem_st32(tmem + lrow, o);
                    else tmem_st16(tmem + lrow, reinterpret_cast<const uint32_t*>(o));
                    tmem_wait_st();
                }
            }
            uint32_t w[NR / 2];
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
                const float x = ex2(z[r] + nm[r]), y = ex2(z[r + 1] + nm[r + 1]);
                l[r] += x;
                l[r + 1] += y;
                w[r / 2] = pack2<OT>(x, y);
            }
            if (j >= 2 && !(ok = warp_wait(pv_done(b), ((j >> 1) - 1) & 1, abort_flag, p.err, 14))) break;
            uint8_t* row = sm + L::P + b * kSeg;
#pragma unroll
            for (int v = 0; v < NR / 8; ++v)
                *reinterpret_cast<uint4*>(row + swz128(threadIdx.x, v)) =
                    make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(b));
        }
        // -------------------------------------------------------- epilogue
        if (ok) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float v = l[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
                if (lane == 0) m_part[warp * NR + r] = v;
            }
            ok = join();
        }
        const bool record = parts > 1;
        if (ok && (int)threadIdx.x < rows) {
            const int r = threadIdx.x;
            const float sum = (m_part[r] + m_part[NR + r]) + (m_part[2 * NR + r] + m_part[3 * NR + r]);
            m_inv[r] = record ? 1.f : sum == 0.f ? 0.f : p.v_scale / sum;
            if (p.max_parts > 1) {
                float m = 0.f;                                 // nm[r], r this thread's
#pragma unroll
                for (int k = 0; k < NR; ++k)
                    if (k == r) m = SHIFT - nm[k];
                // l = -1 marks a row that needs no join
                p.ws_ml[out_row(r) * p.max_parts + part] = make_float2(m, record ? sum : -1.f);
            }
        }
        if (ok) ok = join() && warp_wait(pv_done((nt - 1) & 1), ((nt - 1) >> 1) & 1, abort_flag, p.err, 15);
        const int d = threadIdx.x;                             // this thread's dim
        if (ok && warp * 32 < D) {
            tc_fence_after();
            float o[NR];
            if constexpr (NR == 32) tmem_ld32(tmem + lrow, o);
            else tmem_ld16(tmem + lrow, o);
            tmem_wait_ld();
            if (dirty[1] >= 0) {                               // values were taken out of V
                const int ka = max(lo_c, kb + dirty[0] * kBN);
                const int kz = min(hi_c, kb + dirty[1] * kBN + kBN - 1);
                for (int k = ka; k <= kz; ++k) {
                    if (!masked((k - kb) >> 7)) {              // this tile kept its values
                        k = kb + ((k - kb) | (kBN - 1));
                        continue;
                    }
                    const int id = p.block_tables[(size_t)s * p.MB + (k >> p.log2bs)];
                    if (id < 0 || (long long)id >= p.NB) continue;
                    const float y = cache_value<FP8 ? (int)PA_FP8_E4M3 : QT>(
                        p.v_cache, (((size_t)id * p.bs + (k & (p.bs - 1))) * (p.Hq / p.G) + g) * D + d);
                    if (isfinite(y)) continue;
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (k >= m_lo[r] && k <= m_hi[r]) o[r] += y;
                }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                if (r >= rows) continue;
                if (record) p.ws_o[(out_row(r) * p.max_parts + part) * D + d] = o[r];
                else store_out<QT>(p.out, out_row(r) * D + d, o[r] * m_inv[r]);
            }
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == 5) {
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
