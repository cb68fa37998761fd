// Host side of pa_prefill_scored: argument checks, the split of the keys, the
// workspace and the launch.  The kernels are in prefill_scored.cuh.
#include "prefill_scored.h"

#include <algorithm>
#include <cmath>

#include "pa_internal.h"
#include "tma_host.h"

using pa::clear_error;
using pa::fail;

namespace {

constexpr int kRows = 128, kKeys = 128;      // rows and keys of a tile

// Tokens the key tiles of one query tile pair cover, as the workspace counts
// them: the window of all new tokens, or everything.  Where a prefix lets a row
// see more, the last part takes what is left.
int64_t span_of(int max_query_len, int max_ctx, int window) {
    if (window <= 0) return max_ctx;
    return std::min<int64_t>(max_ctx, (int64_t)window + max_query_len);
}

int64_t parts_of(int max_query_len, int max_ctx, int window, int partition) {
    if (partition == 0) return 1;
    return std::max<int64_t>(1, (span_of(max_query_len, max_ctx, window) + partition - 1) / partition);
}

// Columns of the few-row kernel that hold the rows of a kv head, 0: too many.
int rows_of(int max_query_len, int G) {
    const int64_t rows = (int64_t)max_query_len * G;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 0;
}

pa_status check_sizes(int max_query_len, int max_ctx, int window, int partition) {
    if (max_query_len < 0 || max_ctx < 0 || window < 0 || partition < 0)
        return fail(PA_ERR_INVALID_ARG, "negative size");
    if (partition % kKeys) return fail(PA_ERR_INVALID_ARG, "partition must be a multiple of %d", kKeys);
    return PA_OK;
}

}  // namespace

extern "C" pa_status pa_prefill_scored_suggest_partition(int S, int Hq, int Hkv, int max_query_len,
                                                         int max_ctx, int window, int* partition) {
    clear_error();
    if (!partition || S < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv)
        return fail(PA_ERR_INVALID_ARG, "bad sizes");
    const pa_status st = check_sizes(max_query_len, max_ctx, window, 0);
    if (st) return st;
    *partition = 0;
    const int64_t span = span_of(max_query_len, max_ctx, window);
    if (S == 0 || max_query_len == 0 || span <= 2 * kKeys) return PA_OK;
    // The CTAs of a part run in waves of one per SM, each with about 10 us besides its
    // key tiles (its first loads, its last stores) and 1.2 (few rows) or 3 us a tile;
    // a second kernel joins the parts.  Sequences of a batch are taken to be 0.6 of the
    // longest on average.  Measured against it: 16 sequences of 2k-32k tokens, 8 new,
    // 8 kv heads: 4 parts 188 us, 8 parts 199, 32 parts 304; one of 9.7k: 10 parts 23,
    // 20 parts 31; 16 of 0.2k-2k: one part 30, two 37.
    const bool few = rows_of(max_query_len, Hq / Hkv) != 0;
    const int64_t rows = (int64_t)max_query_len * (Hq / Hkv);
    const double ctas = (double)S * Hkv * (few ? 1 : (rows + 2 * kRows - 1) / (2 * kRows));
    const double fill = ctas * (0.6 + 0.4 / S) / 148.0, tile_us = few ? 1.2 : 3.0;
    const int64_t tiles = (span + kKeys - 1) / kKeys;
    const int64_t most = std::min<int64_t>(tiles / 4, (int64_t)(8.0 / fill) + 1);
    double best = 0.0;
    for (int64_t parts = 1; parts <= most || parts == 1; ++parts) {
        const int64_t per = (tiles + parts - 1) / parts;
        const double us = std::max(1.0, fill * (double)parts + 0.5) * (10.0 + tile_us * (double)per) + (parts > 1 ? 4.0 : 0.0);
        if (parts > 1 && us >= best) continue;
        best = us;
        *partition = parts > 1 ? (int)(per * kKeys) : 0;
    }
    return PA_OK;
}

extern "C" pa_status pa_prefill_scored_workspace_size(int S, int T, int Hq, int D, int max_query_len,
                                                      int max_ctx, int window, int partition,
                                                      size_t* bytes) {
    clear_error();
    if (!bytes || S < 0 || T < 0 || Hq <= 0 || D <= 0) return fail(PA_ERR_INVALID_ARG, "bad sizes");
    const pa_status st = check_sizes(max_query_len, max_ctx, window, partition);
    if (st) return st;
    const int64_t parts = parts_of(max_query_len, max_ctx, window, partition);
    *bytes = 0;
    if (S == 0 || T == 0 || parts == 1) return PA_OK;
    const unsigned __int128 need =
        (unsigned __int128)T * (unsigned)Hq * (unsigned __int128)parts * (sizeof(float2) + sizeof(float) * (unsigned)D);
    if (need > ((unsigned __int128)1 << 60)) return fail(PA_ERR_INVALID_ARG, "workspace size overflows");
    *bytes = (size_t)need + 16;              // the records start at a 16-byte boundary
    return PA_OK;
}

extern "C" pa_status pa_prefill_scored(
    void* out, const void* q, pa_dtype q_dt, const void* key_cache, const void* value_cache,
    pa_dtype cache_dt, const int32_t* block_tables, int MB, const int32_t* context_lens,
    const int32_t* query_start, int S, int T, int Hq, int Hkv, int D, int bs, int64_t NB,
    int max_query_len, int max_ctx, float scale, float k_scale, float v_scale, float softcap,
    const float* slopes, int window, const int32_t* key_start, const int32_t* prefix_lens,
    int partition, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_prefill_scored");
    clear_error();
    if (!pa::valid_dtype(q_dt) || !pa::valid_dtype(cache_dt))
        return fail(PA_ERR_INVALID_ARG, "unknown dtype");
    const bool fp8 = cache_dt == PA_FP8_E4M3;
    if ((q_dt != PA_F16 && q_dt != PA_BF16) || (!fp8 && q_dt != cache_dt))
        return fail(PA_ERR_UNSUPPORTED, "q is f16 or bf16, the cache of the same type or fp8");
    if (D != 64 && D != 128) return fail(PA_ERR_UNSUPPORTED, "head size %d (64 or 128)", D);
    if (fp8 && D != 128) return fail(PA_ERR_UNSUPPORTED, "an fp8 cache needs head size 128");
    if (bs != 8 && bs != 16 && bs != 32) return fail(PA_ERR_UNSUPPORTED, "block size %d", bs);
    if (S < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || MB < 0 || NB <= 0)
        return fail(PA_ERR_INVALID_ARG, "bad sizes");
    const int G = Hq / Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16)
        return fail(PA_ERR_UNSUPPORTED, "group size %d (1, 2, 4, 8 or 16)", G);
    pa::ScoreOpts o;
    o.softcap = softcap;
    o.slopes = slopes;
    o.window = window;
    o.key_start = key_start;
    // with a cap the kernel works on u = 4 z / softcap
    float sl, cap_log2;
    pa_status st = pa::check_score_opts(o, scale, k_scale, 4.0, &sl, &cap_log2);
    if (!st) st = check_sizes(max_query_len, max_ctx, window, partition);
    if (st) return st;
    if (!std::isfinite(scale) || !(scale > 0.f))
        return fail(PA_ERR_INVALID_ARG, "scale must be finite and positive");
    if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
        return fail(PA_ERR_INVALID_ARG, "scales must be finite and > 0");
    if (!fp8 && (k_scale != 1.f || v_scale != 1.f))
        return fail(PA_ERR_INVALID_ARG, "k_scale / v_scale apply to fp8 caches only");
    // key indices past a tile's end stay within an int
    if (max_ctx > (1 << 30)) return fail(PA_ERR_UNSUPPORTED, "max_ctx %d (2^30 at most)", max_ctx);
    if (S == 0 || T == 0 || max_query_len == 0) return PA_OK;
    if (MB == 0) return fail(PA_ERR_INVALID_ARG, "MB == 0 with new tokens");
    if (!out || !q || !key_cache || !value_cache || !block_tables || !context_lens || !query_start)
        return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (!pa::aligned16(out) || !pa::aligned16(q) || !pa::aligned16(key_cache) ||
        !pa::aligned16(value_cache))
        return fail(PA_ERR_INVALID_ARG, "out, q and the caches must be 16-byte aligned");
    // few rows of a kv head: the kernel whose MMA columns are the queries
    const int few = rows_of(max_query_len, G);
    const int TQ = (few ? few : kRows) / G;
    const int64_t n_pairs = few ? 1 : ((int64_t)max_query_len + 2 * TQ - 1) / (2 * TQ);
    const int64_t parts = parts_of(max_query_len, max_ctx, window, partition);
    // as many pair slots per group as there are pairs: a CTA that only exits
    // would hold a whole SM's shared memory for a moment
    const int pair_group = (int)std::min<int64_t>(n_pairs, ps::kPairGroup);
    const int64_t groups = (n_pairs + pair_group - 1) / pair_group;
    if (S > 65535 || groups > 65535 || (int64_t)Hkv * pair_group * parts > 0x7fffffffLL ||
        (int64_t)max_query_len * Hq > 0x7fffffffLL)
        return fail(PA_ERR_UNSUPPORTED, "grid too large (S %d, %lld parts)", S, (long long)parts);
    if (NB > 0x7fffffffLL) return fail(PA_ERR_INVALID_ARG, "NB must fit int32 block ids");
    size_t need = 0;
    st = pa_prefill_scored_workspace_size(S, T, Hq, D, max_query_len, max_ctx, window, partition, &need);
    if (st) return st;
    if (need && (!workspace || workspace_bytes < need || !pa::aligned16(workspace)))
        return fail(PA_ERR_INVALID_ARG, "workspace needs %zu bytes, 16-byte aligned (got %zu)", need,
                    workspace_bytes);

    CUtensorMap mq, mk, mv;
    if ((st = pa::make_rows_map(&mq, q, q_dt, T, Hq, D, G, TQ))) return st;
    if ((st = pa::make_cache_map(&mk, key_cache, cache_dt, NB, bs, Hkv, D))) return st;
    if ((st = pa::make_cache_map(&mv, value_cache, cache_dt, NB, bs, Hkv, D))) return st;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;

    ps::Params p = {};
    p.out = out;
    p.v_cache = value_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.key_start = key_start;
    p.prefix_lens = prefix_lens;
    p.slopes = slopes;
    p.err = err;
    p.NB = NB;
    p.T = T;
    p.Hq = Hq;
    p.G = G;
    p.log2G = __builtin_ctz((unsigned)G);
    p.TQ = TQ;
    p.MB = MB;
    p.bs = bs;
    p.log2bs = __builtin_ctz((unsigned)bs);
    p.max_qlen = max_query_len;
    p.max_ctx = max_ctx;
    p.n_pairs = (int)n_pairs;
    p.pair_group = pair_group;
    p.window = window;
    p.part_tiles = partition / kKeys;
    p.max_parts = (int)parts;
    p.sl = sl;
    p.cap_log2 = cap_log2;
    p.v_scale = v_scale;
    p.ws_ml = static_cast<float2*>(workspace);
    const size_t records = (size_t)T * Hq * (size_t)parts;
    p.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (records * sizeof(float2) + 15) / 16 * 16);

    ps::Launch a;
    a.mq = &mq;
    a.mk = &mk;
    a.mv = &mv;
    a.p = &p;
    a.few = few;
    a.grid = dim3((unsigned)(Hkv * pair_group * parts), (unsigned)S, (unsigned)groups);
    a.stream = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (few)
        e = fp8 ? (q_dt == PA_BF16 ? ps::launch_few_fp8_q_bf16(a, D) : ps::launch_few_fp8_q_f16(a, D))
                : (q_dt == PA_BF16 ? ps::launch_few_bf16(a, D) : ps::launch_few_f16(a, D));
    else
        e = fp8 ? (q_dt == PA_BF16 ? ps::launch_fp8_q_bf16(a, D) : ps::launch_fp8_q_f16(a, D))
                : (q_dt == PA_BF16 ? ps::launch_bf16(a, D) : ps::launch_f16(a, D));
    if (e != cudaSuccess) return pa::cuda_fail(e, "scored prefill launch");
    return PA_OK;
}
