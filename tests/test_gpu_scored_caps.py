"""Caps far above the scores: an error goes with the score, not with the cap."""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc
import test_gpu_decode_scored as dec
import test_gpu_prefill_scored as chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield


# new tokens of a sequence: the few-row kernel, one query tile, two
KERNELS = {"few": [8, 3], "one_tile": [30, 16], "two_tiles": [90, 33]}


CAPS = [50.0, 1e3, 1e4, 1e6, 1e9, 1e20, 1e32]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("Hq,Hkv,D,dt,cdt", [(4, 2, 64, "f32", "f32"), (8, 2, 128, "f32", "f32"),
                                             (8, 2, 128, "bf16", "bf16"), (8, 4, 128, "f16", "fp8"),
                                             (4, 2, 256, "f16", "f16"), (16, 1, 64, "f16", "f16")])
def test_caps_above_the_scores_decode(cap, Hq, Hkv, D, dt, cdt):
    """A cap far above a score changes little of it: errors go with the score, not the cap."""
    c = dec.decode([300, 33, 120], Hq, Hkv, D, 16, dt, cdt, softcap=cap, seed=int(D))
    want = sc.oracle(c)
    for part in (0, 64):
        sc.check(c, dec.run(c, part), f"cap {cap} partition {part}", want)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("kernel", sorted(KERNELS))
@pytest.mark.parametrize("dt,cdt,D", [("bf16", "bf16", 128), ("f16", "f16", 64), ("bf16", "fp8", 128),
                                      ("f16", "fp8", 128)])
def test_caps_above_the_scores_chunk(cap, kernel, dt, cdt, D):
    c = sc.make([700, 250], KERNELS[kernel], 8, 2, D, 16, dt, cdt, softcap=cap, seed=D)
    want = sc.oracle(c)
    for part in (0, 256):
        sc.check(c, chunk.run(c, part), f"cap {cap} partition {part}", want)


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("kernel", sorted(KERNELS) + ["decode"])
def test_small_scores_beside_capped_ones(kernel, alibi):
    """Rows of one tile from a millionth of the cap to far above it."""
    cap = 1e5 if kernel == "decode" else 1e6
    if kernel == "decode":
        c = dec.decode([400] * 12, 8, 2, 128, 16, "f16", "f16", softcap=cap, alibi=alibi, seed=7)
    else:
        c = sc.make([700, 250], KERNELS[kernel], 8, 2, 128, 16, "f16", "f16", softcap=cap, alibi=alibi, seed=7)
    T = c["q"].shape[0]
    low = -2 if kernel == "decode" else -3
    size = torch.logspace(low, 4, T)[torch.randperm(T, generator=torch.Generator().manual_seed(7))]
    c["q"] = (c["q"].float() * size[:, None, None]).clamp(-6e4, 6e4).half()
    c["scale"] = cap / 100
    # keys along one direction, so that scores differ by what the small rows feel
    c["kc"] = torch.where(torch.isnan(c["kc"]), c["kc"], c["kc"] * 0.01)
    want = sc.oracle(c)
    run = dec.run if kernel == "decode" else chunk.run
    for part in (0, 128):
        sc.check(c, run(c, part), f"partition {part}", want)
