"""Scores' factors near the ends of fp32, on 8-bit caches."""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc
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


@pytest.mark.parametrize("kernel", sorted(KERNELS))
@pytest.mark.parametrize("softcap", [0.0, 10.0])
def test_queries_and_scales_near_nothing(kernel, softcap):
    """Factors whose product is below fp32's range: every score is zero, masks hold."""
    c = sc.make([300, 10], KERNELS[kernel], 8, 2, 128, 16, "bf16", "fp8", window=100, softcap=softcap, seed=8)
    c["q"] = (c["q"].double() * 2.0 ** -126).to(torch.bfloat16)
    c["scale"] = 1e-6
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, chunk.run(c, part), f"partition {part}", want)


@pytest.mark.parametrize("kernel", sorted(KERNELS))
@pytest.mark.parametrize("scale", [1e-39, 1.4e-45])
def test_scales_below_the_normal_numbers(kernel, scale):
    c = sc.make([300, 10], KERNELS[kernel], 8, 2, 128, 16, "f16", "fp8", window=100, seed=8)
    c["scale"], c["k_scale"] = scale, 1e-3
    want = sc.oracle(c)
    for part in (0, 128):
        sc.check(c, chunk.run(c, part), f"partition {part}", want)


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_infinite_queries_on_an_8_bit_cache(kernel):
    """A query row with an infinite and large finite elements: its scores are infinite, the cap's."""
    c = sc.make([300, 10], KERNELS[kernel], 8, 2, 128, 16, "bf16", "fp8", softcap=3.0, seed=9)
    codes = c["kc"].view(torch.uint8)
    codes[..., 5] = torch.where(codes[..., 5] & 0x7F == 0, torch.full_like(codes[..., 5], 0x30), codes[..., 5])
    c["q"][1, :, :] = 1e6
    c["q"][1, :, 5] = float("inf")
    c["q"][2, 3, 5] = -float("inf")
    want = sc.oracle(c)
    assert torch.isfinite(want.out).all()
    for part in (0, 128):
        sc.check(c, chunk.run(c, part), f"partition {part}", want)
