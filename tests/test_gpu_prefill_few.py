"""GPU parity of chunk attention with few query rows a kv head (at most 32: the
kernel of pa_prefill_scored whose MMA columns are the queries) against the 64-bit
oracle, with everything that no query may see poisoned."""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc
from test_gpu_prefill_scored import MODS, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield


def few(L, G):
    """Chunk lengths up to L, all of which fit the kernel's columns."""
    assert L * G <= 32
    return [L, 1, max(1, L - 1), L, 1, L, (L + 1) // 2, L]


CACHED = [0, 3, 200, 127, 130, 1500, 64, 700]


@pytest.mark.parametrize("mod", sorted(MODS))
@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,cdt,L", [
    (8, 2, 128, 16, "bf16", "bf16", 8), (2, 2, 128, 16, "f16", "f16", 32),
    (16, 1, 64, 32, "bf16", "bf16", 1), (8, 4, 64, 8, "f16", "f16", 15), (8, 1, 128, 8, "bf16", "bf16", 4),
    (8, 4, 128, 32, "bf16", "fp8", 7), (8, 2, 128, 16, "f16", "fp8", 4), (16, 1, 128, 8, "bf16", "fp8", 2),
    (1, 1, 128, 16, "bf16", "fp8", 30), (1, 1, 64, 16, "bf16", "bf16", 17), (32, 8, 128, 32, "bf16", "fp8", 8),
])
def test_modifications(mod, Hq, Hkv, D, bs, dt, cdt, L):
    c = sc.make(CACHED, few(L, Hq // Hkv), Hq, Hkv, D, bs, dt, cdt, seed=Hq + D + bs + L, **MODS[mod])
    want = sc.oracle(c)
    for part in (0, 128, 384):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 300])
def test_window_edges(window, cdt):
    c = sc.make([0, 127, 128, 129, 400, 31], [8, 1, 2, 8, 5, 7], 8, 2, 128, 16, "bf16", cdt,
                window=window, seed=window)
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt,bs", [("bf16", 16), ("bf16", 8), ("fp8", 32)])
@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("alibi", [False, True])
def test_documents_and_prefixes(cdt, bs, prefix, alibi):
    cached, new = [0, 90, 300, 5, 1000], [8, 7, 8, 1, 3]
    ks = []
    for c_, l in zip(cached, new):
        ks += [c_ + r + 1 if r == 2 else (c_ + r) // 70 * 70 for r in range(l)]
    pl = [8, 0, 320, -7, 10 ** 9] if prefix else None
    c = sc.make(cached, new, 8, 2, 128, bs, "bf16", cdt, alibi=alibi, softcap=0.0 if alibi else 30.0,
                key_start=ks, prefix_lens=pl, seed=5)
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt", ["bf16", "f16", "fp8"])
def test_rows_that_see_nothing(cdt):
    dt = "bf16" if cdt == "fp8" else cdt
    c = sc.make([0, 400], [5, 6], 4, 2, 128, 16, dt, cdt, key_start=[10 ** 6] * 11, seed=1)
    for part in (0, 128):
        assert (run(c, part) == 0).all()
    ks = [10 ** 6] * 11
    ks[2], ks[10] = 0, -3
    c = sc.make([0, 400], [5, 6], 4, 2, 128, 16, dt, cdt, key_start=ks, seed=1)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}")


@pytest.mark.parametrize("cdt,bad", [("bf16", float("nan")), ("bf16", float("inf")),
                                     ("f16", -float("inf")), ("f16", float("nan")), ("fp8", float("nan"))])
@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_values_reach_the_rows_that_see_them_only(cdt, bad, D):
    if cdt == "fp8" and D == 64:
        D = 128
    dt = "bf16" if cdt == "fp8" else cdt
    cached, new = [150, 700], [8, 6]
    for window in (0, 120):
        c = sc.make(cached, new, 8, 2, D, 16, dt, cdt, window=window, seed=2)
        for s, t, d in ((0, 31, 5), (0, 40, 17), (0, 151, 60), (0, 157, 61), (1, 640, 1),
                        (1, 705, 63), (1, 583, 40)):
            if window and t < cached[s] - window + 1:
                continue
            blk = int(c["tables"][s, t // 16])
            if cdt == "fp8":
                sc.poison(c["vc"], blk, t % 16, 1, d)
            else:
                c["vc"][blk, t % 16, 1, d] = bad
        want = sc.oracle(c)
        assert not torch.isfinite(want.out).all() and torch.isfinite(want.out).any()
        for part in (0, 128):
            sc.check(c, run(c, part), f"window {window} partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt", ["bf16", "fp8"])
def test_a_nan_key_reaches_the_rows_that_see_it_only(cdt):
    c = sc.make([200], [8], 8, 2, 128, 16, "bf16", cdt, softcap=7.0, window=60, seed=3)
    t = 203
    sc.poison(c["kc"], int(c["tables"][0, t // 16]), t % 16, 0)
    want = sc.oracle(c)
    assert torch.isnan(want.out).sum() == 5 * 4 * 128
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)


@pytest.mark.parametrize("softcap", [0.5, 5.0, 50.0])
def test_caps_from_the_fit_to_saturation(softcap):
    c = sc.make([900], [16], 4, 2, 128, 16, "bf16", "bf16", softcap=softcap, seed=4)
    c["q"] *= torch.logspace(-3, 3, 16)[:, None, None].to(c["q"].dtype)
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_growing_scores_raise_the_reference_in_every_tile():
    c = sc.make([2000], [4], 4, 2, 128, 16, "f16", "f16", seed=4)
    grow = torch.linspace(-20, 20, 2004)
    c["q"][:] = 0
    c["q"][:, :, 0] = 11.0
    for t in range(2004):
        c["kc"][int(c["tables"][0, t // 16]), t % 16, :, 0] = grow[t]
    c["q"][:, 1, 0] = -11.0
    want = sc.oracle(c)
    for part in (0, 256):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_large_and_negative_slopes():
    c = sc.make([500], [8], 4, 4, 128, 16, "bf16", "bf16", alibi=True, prefix_lens=[506], seed=4, q_scale=10.0)
    c["slopes"] = torch.tensor([1e30, 1e-30, -0.01, 0.0])
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_infinite_scores():
    c = sc.make([300], [4], 4, 4, 128, 16, "bf16", "bf16", softcap=3.0, seed=3)
    c["kc"][int(c["tables"][0, 1]), 3, :, 0] = float("inf")
    c["q"][:, :, 0] = 1.0
    sc.check(c, run(c), "inf")


@pytest.mark.parametrize("exponent", [-90, -20, 60, 100])
def test_queries_of_any_size_on_an_8_bit_cache(exponent):
    c = sc.make([200], [8], 8, 2, 128, 16, "bf16", "fp8", seed=6)
    c["q"] = (c["q"].double() * 2.0 ** exponent).to(torch.bfloat16)
    c["q"][3] = 0
    c["scale"] *= 2.0 ** -exponent
    sc.check(c, run(c), str(exponent))


def test_bad_pages_and_rows_behind():
    c = sc.make([600, 50], [5, 3], 8, 2, 128, 16, "bf16", "fp8", window=300, seed=12)
    for part in (0, 128):
        good = run(c, part)
        assert pa.pa_device_status() == 0
        for bad_id in (10 ** 6, -1, 2 ** 31 - 1):
            bad = dict(c, tables=c["tables"].clone())
            bad["tables"][0, 30] = bad_id
            got = run(bad, part)
            assert pa.pa_device_status() == pa.PA_DEV_BAD_BLOCK
            assert torch.isfinite(got).all() and torch.equal(got[5:], good[5:])
        big = dict(c, q=torch.cat([c["q"], c["q"][:2]]))
        out = torch.full_like(big["q"], 7.0).cuda()
        got = run(big, part, out=out)
        assert torch.equal(got[:8], good) and (got[8:] == 7).all()
        bad = dict(c, lens=torch.tensor([605, 2], dtype=torch.int32))
        out = torch.full_like(c["q"], 7.0).cuda()
        got = run(bad, part, out=out)
        assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT
        assert torch.equal(got[:5], good[:5]) and (got[5:] == 7).all()


def test_captured_replayed_and_repeated():
    c = sc.make([3000, 64, 5], [8, 1, 3], 8, 2, 128, 16, "bf16", "fp8", softcap=10.0, seed=13)
    want = run(c, 512)
    assert torch.equal(run(c, 512), want)
    q, kc, vc, bt, cl, qs = (c[k].cuda() for k in ("q", "kc", "vc", "tables", "lens", "qs"))
    out = torch.empty_like(q)
    ws = torch.empty(pa.pa_prefill_scored_workspace_size(3, 12, 8, 128, 8, c["max_ctx"], 0, 512),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pa.pa_prefill_scored(out, q, kc, vc, bt, cl, qs, 8, c["max_ctx"], c["scale"], softcap=10.0,
                             k_scale=c["k_scale"], v_scale=c["v_scale"], partition=512, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("L", [8, 16, 30])
@pytest.mark.parametrize("cdt", ["bf16", "fp8"])
def test_back_to_back_on_long_contexts(cdt, L):
    """Launches behind each other on more CTAs than the GPU holds, each with many trips
    round its rings (8 new tokens: the few-row kernel; 16 and 30: one query tile whose
    halves take turns): every result the same."""
    g = torch.Generator().manual_seed(L)
    S, Hq, Hkv, D, bs = 12, 16, 4, 128, 16
    n = torch.randint(2000, 24000, (S,), generator=g)
    nblk = (n + bs - 1) // bs
    NB = int(nblk.sum())
    tables = torch.full((S, int(nblk.max())), -1, dtype=torch.int32)
    at = 0
    for s in range(S):
        tables[s, :nblk[s]] = torch.arange(at, at + int(nblk[s]))
        at += int(nblk[s])
    kc, vc = (torch.randn(NB, bs, Hkv, D, device="cuda").mul_(40 if cdt == "fp8" else 1).clamp_(-448, 448)
              .to(sc.DT[cdt]) for _ in range(2))
    q = torch.randn(S * L, Hq, D, device="cuda").bfloat16()
    qs = torch.arange(0, S * L + 1, L, dtype=torch.int32, device="cuda")
    bt, cl = tables.cuda(), n.int().cuda()
    mc = int(n.max())
    ks = 0.025 if cdt == "fp8" else 1.0
    first = {}
    for rep in range(6):
        for part in (0, 1024, 4096):
            nb = pa.pa_prefill_scored_workspace_size(S, S * L, Hq, D, L, mc, 0, part)
            ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
            out = torch.empty_like(q)
            for _ in range(4):
                pa.pa_prefill_scored(out, q, kc, vc, bt, cl, qs, L, mc, D ** -0.5, softcap=20.0, k_scale=ks,
                                     v_scale=ks, partition=part, workspace=ws)
            if part not in first:
                first[part] = out
            assert torch.equal(out, first[part]), (rep, part)
    assert pa.pa_device_status() == 0
    # one sequence against its own keys, in 64 bits
    s, h = 3, 5
    keys = int(n[s])
    rows = tables[s, :int(nblk[s])].long().cuda()
    k, v = (x.view(torch.uint8)[rows].view(x.dtype).float().flatten(0, 1)[:keys, h // 4].double() * ks
            if cdt == "fp8" else x[rows].flatten(0, 1)[:keys, h // 4].double() for x in (kc, vc))
    z = 20.0 * torch.tanh((q[s * L:(s + 1) * L, h].double() @ k.T) * D ** -0.5 / 20.0)
    pos = torch.arange(keys - L, keys, device="cuda")[:, None]
    z = z.masked_fill(torch.arange(keys, device="cuda") > pos, -torch.inf)
    want = torch.softmax(z, -1) @ v
    bound = torch.softmax(z, -1) @ v.abs()
    for part, out in first.items():
        got = out[s * L:(s + 1) * L, h].double()
        # a probability's and the output's rounding (2^-9 and 2^-9 of bf16 at most), fp32 scores
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -12) * bound + 1e-6).all(), part
