"""GPU parity of chunk attention with modified scores (pa_prefill_scored) against
the 64-bit oracle: caps, distance bias, windows, documents and prefixes over the
dtypes, block sizes, head groups and key splits, with everything that no query
may see poisoned.  Tolerances: oracle.scored.Bound; f16 probabilities are kept
2^7 times as large, so those that lose bits weigh below 2^-21 each."""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield


def up(x):
    return None if x is None else x.cuda()


def workspace(c, partition, max_new=None, max_ctx=None):
    T, Hq, D = c["q"].shape
    nb = pa.pa_prefill_scored_workspace_size(len(c["lens"]), T, Hq, D, max_new or c["max_new"],
                                             max_ctx or c["max_ctx"], c["window"], partition)
    return torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda") if nb else None


def run(c, partition=0, stream=None, max_ctx=None, max_new=None, out=None, ws=None):
    q = c["q"].cuda()
    out = torch.full_like(q, float("nan")) if out is None else out
    ws = workspace(c, partition, max_new, max_ctx) if ws is None else ws
    pa.pa_prefill_scored(out, q, c["kc"].cuda(), c["vc"].cuda(), up(c["tables"]), up(c["lens"]),
                         up(c["qs"]), max_new or c["max_new"], max_ctx or c["max_ctx"], c["scale"],
                         softcap=c["softcap"], slopes=up(c["slopes"]), window=c["window"],
                         key_start=up(c["key_start"]), prefix_lens=up(c["prefix_lens"]),
                         k_scale=c["k_scale"], v_scale=c["v_scale"], partition=partition,
                         workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return out


MODS = {"plain": {}, "cap": dict(softcap=5.0), "alibi": dict(alibi=True),
        "cap_alibi": dict(softcap=20.0, alibi=True), "window": dict(window=70),
        "all": dict(softcap=5.0, alibi=True, window=129)}
CACHED = [0, 3, 200, 0, 130, 500, 64]
NEW = [1, 40, 7, 70, 33, 1, 64]


@pytest.mark.parametrize("mod", sorted(MODS))
@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,cdt", [
    (8, 2, 128, 16, "bf16", "bf16"), (2, 2, 128, 16, "f16", "f16"), (16, 1, 64, 32, "bf16", "bf16"),
    (8, 4, 64, 8, "f16", "f16"), (8, 1, 128, 8, "bf16", "bf16"), (8, 4, 128, 32, "bf16", "fp8"),
    (8, 2, 128, 16, "f16", "fp8"), (16, 1, 128, 8, "bf16", "fp8"), (1, 1, 128, 16, "bf16", "fp8"),
    (1, 1, 64, 16, "bf16", "bf16"),
])
def test_modifications(mod, Hq, Hkv, D, bs, dt, cdt):
    c = sc.make(CACHED, NEW, Hq, Hkv, D, bs, dt, cdt, seed=Hq + D + bs, **MODS[mod])
    want = sc.oracle(c)
    for part in (0, 128, 384):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt", ["bf16", "fp8"])
@pytest.mark.parametrize("G", [1, 4, 16])
def test_tile_edges(G, cdt):
    """Chunks at the query tile's size +-1, last keys at a key tile's edge +-1."""
    TQ = 128 // G
    new = [1, TQ - 1, TQ, TQ + 1, 2 * TQ, 2 * TQ + 1, 4 * TQ + 3, 5]
    new = [max(1, x) for x in new]
    cached = [0, 129, 128, 127, 0, 255, 1, 251]
    c = sc.make(cached, new, 2 * G, 2, 128, 16, "bf16", cdt, softcap=9.0, seed=G)
    want = sc.oracle(c)
    for part in (0, 256):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 300])
def test_window_edges(window, cdt):
    c = sc.make([0, 127, 128, 129, 400, 31], [300, 1, 2, 40, 150, 128], 4, 2, 128, 16, "bf16", cdt,
                window=window, seed=window)
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


def documents(cached, new, length):
    out = []
    for c, l in zip(cached, new):
        for r in range(l):
            p = c + r
            out.append(p + 1 if r % 11 == 5 else p // length * length)
    return out


@pytest.mark.parametrize("cdt,bs", [("bf16", 16), ("bf16", 8), ("fp8", 32)])
@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("alibi", [False, True])
def test_documents_and_prefixes(cdt, bs, prefix, alibi):
    cached, new = [0, 90, 300, 5, 0], [200, 130, 65, 1, 31]
    n = [a + b for a, b in zip(cached, new)]
    pl = [n[0], 0, 320, -7, 10 ** 9] if prefix else None
    c = sc.make(cached, new, 8, 2, 128, bs, "bf16", cdt, alibi=alibi, softcap=0.0 if alibi else 30.0,
                key_start=documents(cached, new, 70), prefix_lens=pl, seed=5)
    want = sc.oracle(c)
    for part in (0, 128):
        got = run(c, part)
        sc.check(c, got, f"partition {part}", want)
        if not prefix:
            r = torch.tensor([r % 11 == 5 for l in new for r in range(l)])
            assert (got[r.cuda()] == 0).all()
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("cdt", ["bf16", "f16", "fp8"])
def test_rows_that_see_nothing(cdt):
    dt = "bf16" if cdt == "fp8" else cdt
    cached, new = [0, 100], [50, 300]
    c = sc.make(cached, new, 4, 2, 128, 16, dt, cdt, key_start=[10 ** 6] * 350, seed=1)
    for part in (0, 128):
        assert (run(c, part) == 0).all()
    ks = [10 ** 6] * 350
    ks[20], ks[349] = 0, -3                      # one row each that does
    c = sc.make(cached, new, 4, 2, 128, 16, dt, cdt, key_start=ks, seed=1)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cdt", ["bf16", "f16", "fp8"])
def test_non_finite_values_reach_the_rows_that_see_them_only(cdt, bad):
    """Every place a value may sit: seen by all rows, by some, at both ends of windows."""
    if cdt == "fp8" and bad == bad:
        pytest.skip("E4M3 has no infinity")
    dt = "bf16" if cdt == "fp8" else cdt
    cached, new = [150, 700], [300, 6]
    for window in (0, 120):
        c = sc.make(cached, new, 8, 2, 128, 16, dt, cdt, window=window, seed=2)
        for s, t, d in ((0, 3, 5), (0, 200, 17), (0, 449, 60), (0, 300, 100), (0, 301, 101),
                        (1, 640, 1), (1, 705, 127), (1, 588, 40)):
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
    c = sc.make([100], [200], 8, 2, 128, 16, "bf16", cdt, softcap=7.0, window=60, seed=3)
    t = 180
    sc.poison(c["kc"], int(c["tables"][0, t // 16]), t % 16, 0)
    want = sc.oracle(c)
    assert torch.isnan(want.out).sum() == 60 * 4 * 128
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)


@pytest.mark.parametrize("softcap", [0.5, 5.0, 50.0])
def test_caps_from_the_fit_to_saturation(softcap):
    """Scores far below, about and far above the cap, in one tile and apart."""
    c = sc.make([300], [100], 4, 2, 128, 16, "bf16", "bf16", softcap=softcap, seed=4)
    c["q"] *= torch.logspace(-3, 3, 100)[:, None, None].to(c["q"].dtype)
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)


@pytest.mark.parametrize("dt,cdt,D", [("bf16", "bf16", 128), ("f16", "f16", 64), ("f16", "fp8", 128)])
@pytest.mark.parametrize("softcap", [5.0, 12.0, 25.0])
def test_caps_over_whole_tiles(softcap, dt, cdt, D):
    """Products of about +-8 in most tiles of 128 keys, few of which a mask meets: with the
    middle cap |u| = 4 z / c is at most 4 but above 2, with the others beyond and below."""
    c = sc.make([1100, 700], [70, 129], 8, 2, D, 16, dt, cdt, softcap=softcap, seed=11)
    want = sc.oracle(c)
    for part in (0, 256):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_large_and_negative_slopes():
    c = sc.make([500], [60], 4, 4, 128, 16, "bf16", "bf16", alibi=True, prefix_lens=[540], seed=4,
                q_scale=10.0)
    c["slopes"] = torch.tensor([1e30, 1e-30, -0.01, 0.0])
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)


@pytest.mark.parametrize("exponent", [-90, -20, 60, 100])
def test_queries_of_any_size_on_an_8_bit_cache(exponent):
    """bf16 queries beyond f16's range keep their bits (each row by its own power of two)."""
    c = sc.make([200], [40], 8, 2, 128, 16, "bf16", "fp8", seed=6)
    c["q"] = (c["q"].double() * 2.0 ** exponent).to(torch.bfloat16)
    c["q"][3] = 0
    c["scale"] *= 2.0 ** -exponent
    sc.check(c, run(c), str(exponent))


def test_long_context_split():
    c = sc.make([20000, 12345, 0], [5, 1, 3], 8, 2, 128, 16, "bf16", "fp8", softcap=30.0, seed=6)
    want = sc.oracle(c)
    for part in (0, 512, 4096, pa.pa_prefill_scored_suggest_partition(3, 8, 2, 5, 20005, 0)):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_larger_bounds_than_the_batch():
    c = sc.make([100, 50], [30, 1], 8, 2, 64, 16, "f16", "f16", seed=7)
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, run(c, part, max_ctx=5000, max_new=700), f"partition {part}", want)


def test_agrees_with_pa_prefill():
    c = sc.make([300, 0], [200, 77], 8, 2, 128, 16, "bf16", "bf16", seed=8)
    q = c["q"].cuda()
    out = torch.empty_like(q)
    pa.pa_prefill(out, q, c["kc"].cuda(), c["vc"].cuda(), c["tables"].cuda(), c["lens"].cuda(),
                  c["qs"].cuda(), 200, c["scale"])
    want = sc.oracle(c)
    sc.check(c, out, "pa_prefill", want)
    sc.check(c, run(c), "pa_prefill_scored", want)


def test_one_new_token_agrees_with_decode():
    c = sc.make([99, 400, 0], [1, 1, 1], 8, 2, 128, 16, "bf16", "bf16", softcap=10.0, alibi=True,
                window=64, seed=9)
    d = dict(c, decode=True)
    want = sc.oracle(d)
    sc.check(c, run(c), "chunk", want)


def test_rows_behind_the_last_sequence_stay():
    c = sc.make([10, 20], [5, 6], 8, 2, 128, 16, "bf16", "bf16", seed=10)
    want = run(c)
    for part in (0, 128):
        big = dict(c, q=torch.cat([c["q"], c["q"][:4]]))
        out = torch.full_like(big["q"], 7.0).cuda()
        got = run(big, part, out=out)
        assert torch.equal(got[:11], want) and (got[11:] == 7).all()


def test_an_empty_chunk_between_others():
    c = sc.make([10, 20, 5], [5, 0, 9], 8, 2, 128, 16, "bf16", "bf16", prefix_lens=[3, 9, 14], seed=11)
    sc.check(c, run(c), "empty chunk")


def test_bad_pages_and_lengths_are_reported_not_followed():
    c = sc.make([100, 50], [20, 30], 8, 2, 128, 16, "bf16", "bf16", window=20, seed=12)
    good = run(c)
    assert pa.pa_device_status() == 0
    for bad_id in (10 ** 6, -1, 2 ** 31 - 1):
        bad = dict(c, tables=c["tables"].clone())
        bad["tables"][0, 6] = bad_id
        got = run(bad)
        assert pa.pa_device_status() == pa.PA_DEV_BAD_BLOCK
        assert torch.isfinite(got).all() and torch.equal(got[20:], good[20:])
    for what, kw in (("lens", [-3, 80]), ("lens", [19, 80]), ("lens", [10 ** 6, 80]),
                     ("qs", [0, -4, 50]), ("qs", [-2, 20, 50])):
        for part in (0, 128):
            bad = dict(c)
            bad[what] = torch.tensor(kw, dtype=torch.int32)
            run(bad, part)
            assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT, (what, kw)
    bad = dict(c, qs=torch.tensor([0, 20, 51], dtype=torch.int32))       # a row past T
    out = torch.full_like(c["q"], 7.0).cuda()
    got = run(bad, out=out, max_new=64)
    assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT
    assert torch.equal(got[:20], good[:20]) and (got[20:] == 7).all()
    assert torch.equal(run(c), good)


def test_captured_replayed_and_repeated():
    c = sc.make([300, 64, 5], [30, 1, 9], 8, 2, 128, 16, "bf16", "bf16", softcap=10.0, window=200, seed=13)
    want = run(c, 128)
    assert torch.equal(run(c, 128), want)
    q, kc, vc, bt, cl, qs = (c[k].cuda() for k in ("q", "kc", "vc", "tables", "lens", "qs"))
    out = torch.empty_like(q)
    ws = workspace(c, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pa.pa_prefill_scored(out, q, kc, vc, bt, cl, qs, c["max_new"], c["max_ctx"], c["scale"],
                             softcap=10.0, window=200, partition=128, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_streams_at_once():
    a = sc.make([3000, 64], [30, 200], 8, 2, 128, 16, "bf16", "bf16", softcap=10.0, seed=14)
    b = sc.make([100, 2000], [130, 3], 8, 2, 128, 16, "bf16", "fp8", alibi=True, seed=15)
    wa, wb = run(a, 256), run(b, 256)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = []
    for c in (a, b):
        dev.append([c[k].cuda() for k in ("q", "kc", "vc", "tables", "lens", "qs")] + [workspace(c, 256), up(c["slopes"])])
    outs = [torch.zeros_like(d[0]) for d in dev]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, o, st in zip((a, b), dev, outs, streams):
            pa.pa_prefill_scored(o, *d[:6], c["max_new"], c["max_ctx"], c["scale"],
                                 softcap=c["softcap"], slopes=d[7], k_scale=c["k_scale"],
                                 v_scale=c["v_scale"], partition=256, workspace=d[6], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], wa) and torch.equal(outs[1], wb)
