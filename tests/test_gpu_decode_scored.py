"""GPU parity of single-token attention with modified scores (pa_decode_scored)
against the 64-bit oracle: caps, distance bias, windows and first visible keys,
over the dtypes, block sizes, head groups and split sizes, with everything that
no query may see poisoned.  Tolerances: oracle.scored.Bound."""
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
    pa.pa_decode_select(pa.DECODE_DEFAULT)


def run(c, partition=0, stream=None, max_ctx=None, out=None):
    up = lambda x: None if x is None else x.cuda()                      # noqa: E731
    q = c["q"].cuda()
    S, Hq, D = q.shape
    bs = c["kc"].shape[1]
    mc = c["max_ctx"] if max_ctx is None else max_ctx
    nb = pa.pa_decode_scored_workspace_size(S, Hq, D, bs, mc, c["window"], partition)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda") if nb else None
    out = torch.full_like(q, float("nan")) if out is None else out
    pa.pa_decode_scored(out, q, c["kc"].cuda(), c["vc"].cuda(), up(c["tables"]), up(c["lens"]), mc,
                        c["scale"], softcap=c["softcap"], slopes=up(c["slopes"]),
                        window=c["window"], key_start=up(c["key_start"]), k_scale=c["k_scale"],
                        v_scale=c["v_scale"], partition=partition, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return out


def decode(lens, *a, **kw):
    return sc.make([n - 1 if n else 0 for n in lens], [1] * len(lens), *a, decode=True, **kw)


MODS = {"plain": {}, "cap": dict(softcap=5.0), "alibi": dict(alibi=True),
        "cap_alibi": dict(softcap=20.0, alibi=True), "window": dict(window=70),
        "all": dict(softcap=5.0, alibi=True, window=129)}
LENS = [1, 17, 64, 70, 71, 128, 129, 300]


@pytest.mark.parametrize("mod", sorted(MODS))
@pytest.mark.parametrize("Hq,Hkv,D,bs,dt,cdt", [
    (8, 2, 128, 16, "bf16", "bf16"), (32, 8, 128, 16, "bf16", "bf16"),
    (4, 4, 128, 16, "f16", "f16"), (16, 1, 64, 32, "bf16", "bf16"), (8, 4, 64, 8, "f16", "f16"),
    (16, 2, 128, 8, "bf16", "bf16"), (8, 4, 128, 32, "bf16", "fp8"), (8, 2, 128, 16, "f16", "fp8"),
    (16, 1, 128, 8, "bf16", "fp8"), (4, 2, 64, 16, "f32", "f32"), (4, 1, 128, 8, "f32", "f32"),
    (4, 2, 256, 16, "bf16", "bf16"), (2, 2, 256, 32, "f16", "fp8"),
])
def test_modifications(mod, Hq, Hkv, D, bs, dt, cdt):
    c = decode(LENS, Hq, Hkv, D, bs, dt, cdt, seed=Hq + D + bs, **MODS[mod])
    want = sc.oracle(c)
    for part in (0, 64):
        sc.check(c, run(c, part), f"partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("mode", [pa.DECODE_DEFAULT, pa.DECODE_DEFAULT | pa.DECODE_SIMT_ONLY,
                                  pa.DECODE_DEFAULT | pa.DECODE_GROUP_PARTITIONS,
                                  pa.DECODE_DEFAULT | pa.DECODE_ONE_HEAD_PER_CTA,
                                  pa.DECODE_DEFAULT | pa.DECODE_ONE_HEAD_PER_CTA | pa.DECODE_GROUP_PARTITIONS, 0])
def test_kernel_choices(mode):
    pa.pa_decode_select(mode)
    try:
        for cdt in ("bf16", "fp8"):
            c = decode([500, 33, 1000, 256], 16, 4, 128, 16, "bf16", cdt, softcap=8.0, alibi=True,
                       window=300, key_start=[400, 0, 0, 250], seed=mode)
            want = sc.oracle(c)
            for part in (0, 16, 48, 128):
                sc.check(c, run(c, part), f"{cdt} partition {part}", want)
    finally:
        pa.pa_decode_select(pa.DECODE_DEFAULT)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("window", [1, 2, 7, 8, 9, 31, 32, 33, 1000])
def test_window_edges(bs, window):
    lens = [1, 2, 7, 8, 9, 31, 32, 33, 34, 40, 65, 200]
    for cdt in ("bf16", "fp8"):
        c = decode(lens, 8, 4, 128, bs, "bf16", cdt, window=window, seed=window)
        want = sc.oracle(c)
        for part in (0, 32):
            sc.check(c, run(c, part), f"{cdt} {part}", want)
    assert pa.pa_device_status() == 0


def test_first_visible_keys_and_rows_that_see_nothing():
    lens = [40, 40, 40, 40, 40, 0, 300, 300]
    start = [0, 39, 40, 1000, -5, 3, 17, 299]
    for bs in (8, 16):
        c = decode(lens, 8, 2, 128, bs, "bf16", "bf16", key_start=start, seed=1)
        want = sc.oracle(c)
        for part in (0, 32):
            got = run(c, part)
            sc.check(c, got, f"bs {bs} partition {part}", want)
            assert (got[[2, 3, 5]] == 0).all()
    assert pa.pa_device_status() == 0


def test_nan_of_a_visible_key_reaches_its_rows_only():
    c = decode([100, 100], 8, 2, 128, 16, "bf16", "bf16", softcap=10.0, window=50, seed=2)
    t = 70
    sc.poison(c["vc"], int(c["tables"][1, t // 16]), t % 16, 1, 5)
    sc.poison(c["kc"], int(c["tables"][0, t // 16]), t % 16, 0)
    want = sc.oracle(c)
    assert torch.isnan(want.out).sum() == 4 + 4 * 128
    for part in (0, 16):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_infinite_scores_meet_the_cap():
    """A key with an infinite element scores the cap (tanh of infinity is 1)."""
    c = decode([64], 4, 4, 128, 16, "f32", "f32", softcap=3.0, seed=3)
    c["kc"][int(c["tables"][0, 1]), 3, :, 0] = float("inf")
    c["q"][:, :, 0] = 1.0
    sc.check(c, run(c), "inf")


def test_lowest_scores_and_large_biases():
    """Scores and biases at the far ends of fp32: the distant keys weigh nothing."""
    c = decode([3000], 4, 4, 128, 16, "bf16", "bf16", alibi=True, seed=4, q_scale=30.0)
    c["slopes"] = torch.tensor([1e30, 1e-30, -0.01, 0.0])
    c["tables"] = c["tables"].clone()
    sc.check(c, run(c, 256), "biases")


def test_without_modifications_it_is_pa_decode():
    c = decode([700, 33, 1], 16, 4, 128, 16, "bf16", "bf16", seed=5)
    for part in (0, 128):
        got = run(c, part)
        out = torch.empty_like(got)
        nb = pa.pa_decode_workspace_size(3, 16, 128, 700, part)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
        pa.pa_decode(out, c["q"].cuda(), c["kc"].cuda(), c["vc"].cuda(), c["tables"].cuda(),
                     c["lens"].cuda(), 700, c["scale"], partition=part, workspace=ws if nb else None)
        assert torch.equal(out, got)


def test_long_context_split():
    c = decode([20000, 12345], 8, 2, 128, 16, "bf16", "fp8", softcap=30.0, seed=6)
    want = sc.oracle(c)
    for part in (512, 4096):
        sc.check(c, run(c, part), f"partition {part}", want)


def test_rows_outside_the_call_and_bad_values():
    c = decode([100, 50], 8, 2, 128, 16, "bf16", "bf16", window=20, seed=7)
    c["tables"][0, 5] = 10 ** 6                  # a visible block that does not exist
    run(c)
    assert pa.pa_device_status() == pa.PA_DEV_BAD_BLOCK
    c = decode([100, 50], 8, 2, 128, 16, "bf16", "bf16", window=20, seed=7)
    good = run(c)
    bad = dict(c, lens=torch.tensor([-3, 50], dtype=torch.int32))
    got = run(bad)
    assert pa.pa_device_status() == pa.PA_DEV_BAD_CONTEXT
    assert (got[0] == 0).all() and torch.equal(got[1], good[1])


def test_captured_and_replayed():
    c = decode([300, 64, 5], 8, 2, 128, 16, "bf16", "bf16", softcap=10.0, window=200, seed=8)
    want = run(c, 64)
    q, kc, vc, bt, cl = (c[k].cuda() for k in ("q", "kc", "vc", "tables", "lens"))
    out = torch.empty_like(q)
    ws = torch.empty(pa.pa_decode_scored_workspace_size(3, 8, 128, 16, 300, 200, 64),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pa.pa_decode_scored(out, q, kc, vc, bt, cl, 300, c["scale"], softcap=10.0, window=200,
                            partition=64, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    c = decode([30, 20], 8, 2, 128, 16, "bf16", "bf16", seed=9)
    q, kc, vc, bt, cl = (c[k].cuda() for k in ("q", "kc", "vc", "tables", "lens"))
    out = torch.empty_like(q)

    def bad(status="PA_ERR_INVALID_ARG", out=out, q=q, kc=kc, vc=vc, bt=bt, cl=cl, **kw):
        with pytest.raises(pa.PaError) as e:
            pa.pa_decode_scored(out, q, kc, vc, bt, cl, 30, 0.1, **kw)
        assert e.value.status == status, str(e.value)

    bad(softcap=-1.0)
    bad(softcap=float("nan"))
    bad(softcap=float("inf"))
    bad(softcap=1e-44)
    bad(window=-1)
    bad(partition=-1)
    bad(partition=24)
    bad(partition=16)                                     # no workspace
    bad(slopes=torch.ones(4, device="cuda"))
    bad(slopes=torch.ones(8, device="cuda", dtype=torch.float64))
    bad(slopes=torch.ones(8))
    bad(key_start=torch.zeros(3, device="cuda", dtype=torch.int32))
    bad(key_start=torch.zeros(2, device="cuda", dtype=torch.int64))
    bad(out=out[:1])
    bad(out=out.float())
    bad(vc=vc[:2])
    bad(cl=cl[:1])
    bad(k_scale=2.0)
    bad("PA_ERR_UNSUPPORTED", kc=kc.float(), vc=vc.float())
