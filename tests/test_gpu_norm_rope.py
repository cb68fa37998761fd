"""GPU parity of the fused norm + rotation + append against the 64-bit oracle.

Tolerances.  A row's arithmetic is fp32 and each result is rounded once: the
output's half step, plus the fp32 error of what it is made of, |a| + |b|.  The
sum of squares adds 16 products a lane and log2(D / 16) shuffles: 20 half steps,
10 after the root, which itself is within 2 ulp (4 half steps); the division by
D, the eps and three products add 5, the rotation 3: below 32 half steps.
"""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
from oracle import scored

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
      "fp8": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield


def _case(T, Hq, Hkv, D, bs, dt, cdt, norm, rot, interleaved, seed=0, offset=0.0, packed=True,
          P=5000):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)                       # noqa: E731
    qkv = rnd(T, (Hq + 2 * Hkv) * D).to(DT[dt])
    c = {"q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
         "v": qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D), "qkv": qkv}
    NB = (T + bs - 1) // bs + 3
    c["kc"] = rnd(NB, bs, Hkv, D).to(DT[cdt])
    c["vc"] = rnd(NB, bs, Hkv, D).to(DT[cdt])
    c["slots"] = torch.randperm(NB * bs, generator=g)[:T]
    c["slots"][3::7] = -1
    c["qw"] = (1 + 0.3 * rnd(D)).to(DT[dt]) if norm else None
    c["kw"] = (1 + 0.3 * rnd(D)).to(DT[dt]) if norm else None
    c["cs"] = c["pos"] = None
    if rot:
        ang = torch.arange(P, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        c["cs"] = torch.cat((ang.cos(), ang.sin()), 1).float()
        c["pos"] = torch.randint(0, P, (T,), generator=g)
    c.update(eps=1e-6, offset=offset, interleaved=interleaved,
             k_scale=0.02 if cdt == "fp8" else 1.0, v_scale=0.03 if cdt == "fp8" else 1.0,
             dt=dt, cdt=cdt)
    return c


def _gpu(c, in_place=False, stream=None):
    T, Hq, D = c["q"].shape
    Hkv = c["k"].shape[1]
    qkv = c["qkv"].cuda()
    q, k, v = (qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
               qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))
    out = q if in_place else torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    up = lambda x: None if x is None else x.cuda()                      # noqa: E731
    kc, vc = c["kc"].cuda(), c["vc"].cuda()
    pa.pa_norm_rope_append(out, q, k, v, up(c["qw"]), up(c["kw"]), c["eps"], up(c["cs"]),
                           up(c["pos"]), kc, vc, up(c["slots"]), interleaved=c["interleaved"],
                           weight_offset=c["offset"], k_scale=c["k_scale"], v_scale=c["v_scale"],
                           stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), kc.cpu(), vc.cpu()


def _close(got, want, size, dt, what):
    g = scored.stored(got)
    fin = torch.finfo(DT[dt])
    tol = fin.eps / 2 * want.abs() + 32 * 2.0 ** -24 * (1 + fin.eps) * size
    tol = torch.maximum(tol, torch.full_like(tol, fin.smallest_normal * fin.eps))   # subnormal steps
    assert torch.isfinite(g).all(), what
    over = (g - want).abs() - tol
    assert (over <= 0).all(), f"{what}: {float(over.max()):.3g} over the tolerance"


def _check(c, got, what):
    out, kc, vc = got
    want, size = scored.norm_rope(c["q"], c["qw"], c["eps"], c["offset"], c["cs"], c["pos"],
                                  c["interleaved"])
    _close(out, want, size, c["dt"], what + " q")
    kwant, ksize = scored.norm_rope(c["k"], c["kw"], c["eps"], c["offset"], c["cs"], c["pos"],
                                    c["interleaved"])
    Hkv, D = c["k"].shape[1:]
    keep = c["slots"] >= 0
    sl = c["slots"][keep]
    for cache, old, x, xs, sc, name in ((kc, c["kc"], kwant, ksize, c["k_scale"], "k"),
                                        (vc, c["vc"], scored.stored(c["v"]),
                                         0 * scored.stored(c["v"]), c["v_scale"], "v")):
        raw = torch.uint8 if c["cdt"] == "fp8" else {4: torch.int32, 2: torch.int16}[cache.element_size()]
        untouched = torch.ones(cache.shape[0] * cache.shape[1], dtype=torch.bool)
        untouched[sl] = False
        assert torch.equal(cache.view(raw).view(-1, Hkv, D)[untouched],
                           old.view(raw).view(-1, Hkv, D)[untouched]), f"{what} {name}: other slots"
        rows = cache.view(-1, Hkv, D)[sl] if c["cdt"] != "fp8" else \
            cache.view(raw).view(-1, Hkv, D)[sl].view(cache.dtype)
        if c["cdt"] == "fp8":
            s32 = float(torch.tensor(sc, dtype=torch.float32))
            _close(rows, (x[keep] / s32).clamp(-448, 448), xs[keep] / s32 + 2.0 ** -23 * x[keep].abs() / s32,
                   "fp8", f"{what} {name}")
        else:
            _close(rows, x[keep], xs[keep], c["cdt"], f"{what} {name}")


SHAPES = [
    # T, Hq, Hkv, D, bs, in, cache, norm, rot, interleaved
    (1, 8, 2, 128, 16, "bf16", "bf16", True, 128, False),
    (5, 32, 8, 128, 16, "bf16", "bf16", True, 128, False),
    (33, 32, 8, 128, 32, "bf16", "fp8", True, 128, False),
    (7, 3, 3, 64, 8, "f16", "f16", True, 64, False),
    (130, 16, 1, 64, 16, "f16", "fp8", True, 16, True),
    (19, 5, 5, 64, 16, "f32", "f32", True, 32, True),
    (64, 8, 4, 128, 16, "f32", "fp8", True, 128, False),
    (11, 6, 2, 256, 16, "bf16", "bf16", True, 256, False),
    (21, 4, 4, 256, 32, "f16", "f16", True, 64, False),
    (9, 2, 1, 256, 8, "f32", "f32", False, 128, True),
    (2500, 4, 2, 128, 16, "bf16", "bf16", True, 128, False),
    (300, 12, 4, 128, 16, "f16", "f16", False, 112, False),
    (40, 7, 1, 128, 16, "bf16", "fp8", False, 0, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_matches_the_oracle(shape):
    c = _case(*shape, seed=shape[0])
    _check(c, _gpu(c), "out of place")
    _check(c, _gpu(c, in_place=True), "in place")
    assert pa.pa_device_status() == 0


def test_weight_offset_and_far_positions():
    c = _case(50, 8, 2, 128, 16, "bf16", "bf16", True, 128, False, seed=3, offset=1.0, P=200000)
    c["pos"][0], c["pos"][1] = 199999, 0
    _check(c, _gpu(c), "offset")


def test_one_norm_only_and_a_zero_row():
    c = _case(20, 8, 2, 128, 16, "f16", "f16", True, 128, False, seed=4)
    c["kw"] = None
    c["qkv"][5] = 0
    _check(c, _gpu(c), "q norm only")


def test_without_norm_and_rotation_it_is_the_plain_append():
    for dt, cdt in (("bf16", "bf16"), ("f16", "fp8"), ("f32", "f32"), ("f32", "fp8")):
        c = _case(77, 8, 2, 128, 16, dt, cdt, False, 0, False, seed=5)
        out, kc, vc = _gpu(c)
        assert torch.equal(out, c["q"])
        k2, v2 = c["kc"].cuda(), c["vc"].cuda()
        pa.pa_reshape_and_cache(c["k"].contiguous().cuda(), c["v"].contiguous().cuda(), k2, v2,
                                c["slots"].cuda(), c["k_scale"], c["v_scale"])
        assert torch.equal(kc.view(torch.uint8), k2.cpu().view(torch.uint8))
        assert torch.equal(vc.view(torch.uint8), v2.cpu().view(torch.uint8))


@pytest.mark.parametrize("scale", [1.0, 0.02, 3.3e-3, 0.1, 7.0, 1e-17, 3e17, 1e-30, 7e25])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_codes_are_the_plain_append_s_for_any_value_and_scale(dt, scale):
    """Values of every exponent, borders between codes and their neighbours: bit for bit."""
    g = torch.Generator().manual_seed(11)
    T, Hkv, D = 512, 4, 128
    n = T * Hkv * D
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().nan_to_num(448.0)
    mid = (codes[torch.randint(0, 256, (n // 4,), generator=g)] * (1 + torch.randint(-3, 4, (n // 4,), generator=g) * 2.0 ** -5)).double() * scale
    wide = torch.randn(n // 4, generator=g).double() * 2.0 ** torch.randint(-140, 120, (n // 4,), generator=g).double()
    near = torch.randn(n // 2, generator=g).double() * 150 * scale
    x = torch.cat([mid, wide, near]).clamp(-3e38, 3e38).float()
    x[:6] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 448.0 * scale])
    x = x[torch.randperm(n, generator=g)].view(T, Hkv, D).to(DT[dt]).cuda()
    caches = [torch.zeros(T // 16, 16, Hkv, D, device="cuda", dtype=torch.uint8).view(DT["fp8"]) for _ in range(4)]
    slots = torch.arange(T, device="cuda")
    q = torch.zeros(T, 4, D, dtype=x.dtype, device="cuda")
    pa.pa_norm_rope_append(q, q, x, x.flip(0).contiguous(), None, None, 0.0, None, None, caches[0], caches[1],
                           slots, k_scale=scale, v_scale=scale * 0.75)
    pa.pa_reshape_and_cache(x, x.flip(0).contiguous(), caches[2], caches[3], slots, scale, scale * 0.75)
    for a, b in zip(caches[:2], caches[2:]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_bad_slots_and_positions_are_reported_not_followed():
    c = _case(30, 8, 2, 128, 16, "bf16", "bf16", True, 128, False, seed=6)
    c["slots"][:] = torch.randperm(c["kc"].shape[0] * 16, generator=torch.Generator().manual_seed(1))[:30]
    good = _gpu(c)
    assert pa.pa_device_status() == 0
    bad = dict(c, slots=c["slots"].clone(), pos=c["pos"].clone())
    bad["slots"][4] = c["kc"].shape[0] * 16
    out, kc, vc = _gpu(bad)
    assert pa.pa_device_status() == pa.PA_DEV_BAD_SLOT
    assert torch.equal(out, good[0])                       # the query row does not need the slot
    row = int(c["slots"][4])
    assert torch.equal(kc.view(-1, 2, 128)[row], c["kc"].view(-1, 2, 128)[row])
    for p in (-1, 5000, 1 << 40):
        bad = dict(c, pos=c["pos"].clone())
        bad["pos"][9] = p
        out, kc, vc = _gpu(bad)
        assert pa.pa_device_status() == pa.PA_DEV_BAD_POSITION
        assert (out[9] == 7).all() and torch.equal(out[:9], good[0][:9]) and torch.equal(out[10:], good[0][10:])
        row = int(c["slots"][9])
        assert torch.equal(kc.view(-1, 2, 128)[row], c["kc"].view(-1, 2, 128)[row])


def test_captured_and_replayed_on_a_side_stream():
    c = _case(16, 8, 2, 128, 16, "bf16", "bf16", True, 128, False, seed=7)
    want = _gpu(c)
    T, Hq, D = c["q"].shape
    q, k, v = c["q"].contiguous().cuda(), c["k"].contiguous().cuda(), c["v"].contiguous().cuda()
    kc, vc, out = c["kc"].cuda(), c["vc"].cuda(), torch.empty(T, Hq, D, dtype=q.dtype, device="cuda")
    rest = [c[x].cuda() for x in ("qw", "kw", "cs", "pos", "slots")]
    args = (out, q, k, v, rest[0], rest[1], 1e-6, rest[2], rest[3], kc, vc, rest[4])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_norm_rope_append(*args)
    out.fill_(3)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((out, kc, vc), want):
        assert torch.equal(got.cpu(), w)


def test_refusals():
    c = _case(4, 8, 2, 128, 16, "bf16", "bf16", True, 128, False)
    q, k, v, kc, vc, sl, cs, pos = (c[x].cuda() for x in ("q", "k", "v", "kc", "vc", "slots", "cs", "pos"))
    out = torch.empty_like(q)

    def bad(*a, **kw):
        with pytest.raises(pa.PaError) as e:
            pa.pa_norm_rope_append(*a, **kw)
        return e.value.status

    assert bad(out, q, k, v, None, None, 1e-6, cs, pos[:3], kc, vc, sl) == "PA_ERR_INVALID_ARG"
    assert bad(out, q, k, v, None, None, 1e-6, cs, pos, kc, vc, sl[:3]) == "PA_ERR_INVALID_ARG"
    assert bad(out, q, k[:3], v, None, None, 1e-6, cs, pos, kc, vc, sl) == "PA_ERR_INVALID_ARG"
    assert bad(out, q.cpu(), k, v, None, None, 1e-6, cs, pos, kc, vc, sl) == "PA_ERR_INVALID_ARG"
    assert bad(out, q.float(), k, v, None, None, 1e-6, cs, pos, kc, vc, sl) == "PA_ERR_INVALID_ARG"
    assert bad(out, q, k, v, torch.ones(64, device="cuda", dtype=q.dtype), None, 1e-6, cs, pos, kc, vc, sl) == "PA_ERR_INVALID_ARG"
    assert bad(out, q, k, v, None, None, 1e-6, cs[:, :24].contiguous(), pos, kc, vc, sl) == "PA_ERR_UNSUPPORTED"
    assert bad(out, q, k, v, None, None, 1e-6, cs[:, ::2], pos, kc, vc, sl) == "PA_ERR_INVALID_ARG"
    assert bad(out, q, k, v, None, None, 1e-6, cs, pos, kc, vc, sl, k_scale=2.0) == "PA_ERR_INVALID_ARG"
    assert bad(out.transpose(1, 2), q, k, v, None, None, 1e-6, cs, pos, kc, vc, sl) == "PA_ERR_INVALID_ARG"
    # no tokens: nothing to do
    pa.pa_norm_rope_append(out[:0], q[:0], k[:0], v[:0], None, None, 1e-6, cs, pos[:0], kc, vc, sl[:0])
