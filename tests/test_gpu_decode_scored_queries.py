"""bf16 queries of any size on an 8-bit cache, for single tokens: beyond f16's range, below
it, and with infinite elements (as the chunk kernels take them)."""
import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc
import test_gpu_decode_scored as dec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield


SHAPES = [(8, 4, 16), (16, 1, 32), (16, 2, 8), (3, 3, 16), (32, 8, 32)]


@pytest.mark.parametrize("exponent", [-90, -30, -20, 0, 30, 60, 100])
@pytest.mark.parametrize("Hq,Hkv,bs", SHAPES)
def test_queries_of_any_size(exponent, Hq, Hkv, bs):
    c = dec.decode([200, 33, 1, 90], Hq, Hkv, 128, bs, "bf16", "fp8", seed=6, softcap=20.0)
    c["q"] = (c["q"].double() * 2.0 ** exponent).to(torch.bfloat16)
    c["q"][3, 0] = 0
    # rows of their own sizes beside one another
    c["q"][0] *= torch.logspace(0, -4, Hq, base=2.0).to(torch.bfloat16)[:, None]
    c["scale"] *= 2.0 ** -exponent
    want = sc.oracle(c)
    for part in (0, 64):
        sc.check(c, dec.run(c, part), f"{exponent} partition {part}", want)


@pytest.mark.parametrize("Hq,Hkv,bs", SHAPES[:3])
def test_infinite_queries(Hq, Hkv, bs):
    c = dec.decode([200, 33, 90], Hq, Hkv, 128, bs, "bf16", "fp8", seed=9, softcap=3.0)
    codes = c["kc"].view(torch.uint8)
    codes[..., 5] = torch.where(codes[..., 5] & 0x7F == 0, torch.full_like(codes[..., 5], 0x30), codes[..., 5])
    c["q"][1, :, :] = 1e6
    c["q"][1, :, 5] = float("inf")
    c["q"][2, 1, 5] = -float("inf")
    want = sc.oracle(c)
    assert torch.isfinite(want.out).all()
    for part in (0, 64):
        sc.check(c, dec.run(c, part), f"partition {part}", want)
