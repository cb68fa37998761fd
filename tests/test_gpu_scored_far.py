"""The distance bias at positions past fp32's whole numbers, in decode and the chunk kernels."""
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


def far(c, tokens):
    """The same keys behind `tokens` more that no query sees (blocks that do not exist): every
    row's window ends inside the keys there are."""
    bs = c["kc"].shape[1]
    assert 0 < c["window"] <= int((c["lens"] - c["qs"].diff()).min()) + 1
    S = len(c["lens"])
    ahead = torch.full((S, tokens // bs), c["kc"].shape[0] + 7, dtype=torch.int32)
    return dict(c, tables=torch.cat([ahead, c["tables"]], 1), lens=c["lens"] + tokens,
                max_ctx=c["max_ctx"] + tokens,
                key_start=None if c["key_start"] is None else c["key_start"] + tokens)


@pytest.mark.parametrize("tokens", [1 << 24, 20_000_000, 1 << 28])
@pytest.mark.parametrize("kernel", sorted(KERNELS))
@pytest.mark.parametrize("dt,cdt,D", [("bf16", "bf16", 64), ("bf16", "fp8", 128)])
def test_bias_at_far_positions_chunk(tokens, kernel, dt, cdt, D):
    """Distances are exact where positions no longer are in fp32 (from 2^24 on)."""
    new = KERNELS[kernel]
    c = sc.make([101, 64], new, 8, 2, D, 16, dt, cdt, alibi=True, window=48, seed=3)
    c["slopes"] = torch.tensor([0.5, 0.25, 1.0, 2.0, 0.125, 3.0, -0.25, 0.7])
    want = sc.oracle(c)
    f = far(c, tokens)
    for part in (0, 128):
        sc.check(c, chunk.run(f, part), f"{tokens} partition {part}", want)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("tokens", [1 << 24, 20_000_000])
@pytest.mark.parametrize("dt,cdt", [("bf16", "bf16"), ("f32", "f32")])
def test_bias_at_far_positions_decode(tokens, dt, cdt):
    c = dec.decode([101, 65], 8, 4, 64, 16, dt, cdt, alibi=True, window=48, seed=4)
    c["slopes"] = torch.tensor([0.5, 0.25, 1.0, 2.0, 0.125, 3.0, -0.25, 0.7])
    want = sc.oracle(c)
    for part in (0, 16):
        sc.check(c, dec.run(far(c, tokens), part), f"{tokens} partition {part}", want)
    assert pa.pa_device_status() == 0
