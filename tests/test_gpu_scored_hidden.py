"""What stands in keys that a row does not see, or in rows that are not its sequence's,
does not change a bit of it."""
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


def refill(c, keys, value, seed=0):
    """c with other K and V in the given (sequence, token) places: value times noise."""
    g = torch.Generator().manual_seed(seed)
    bs = c["kc"].shape[1]
    out = dict(c, kc=c["kc"].clone(), vc=c["vc"].clone())
    for s, t in keys:
        b = int(c["tables"][s, t // bs])
        if not 0 <= b < c["kc"].shape[0]:
            continue
        for name in ("kc", "vc"):
            x = torch.randn(c["kc"].shape[2:], generator=g) * value
            out[name][b, t % bs] = x.clamp(-448, 448).to(out[name].dtype) if c["cdt"] == "fp8" else x.to(out[name].dtype)
    return out


@pytest.mark.parametrize("cap", [0.0, 2.0, 6.0, 40.0])
@pytest.mark.parametrize("kernel", sorted(KERNELS) + ["decode"])
@pytest.mark.parametrize("dt,cdt", [("bf16", "bf16"), ("f16", "fp8")])
def test_hidden_keys_do_not_change_a_bit(cap, kernel, dt, cdt):
    """Slots past the last token and before every window: zeros or large numbers, alike."""
    cached, new = [300, 77], [1, 1] if kernel == "decode" else KERNELS[kernel]
    c = sc.make(cached, new, 8, 2, 128, 16, dt, cdt, softcap=cap, window=100, seed=10, decode=kernel == "decode")
    n = [int(x) for x in c["lens"]]
    hidden = [(s, t) for s in (0, 1) for t in list(range(max(0, cached[s] - 99))) + list(range(n[s], -(-n[s] // 16) * 16))]
    run = dec.run if kernel == "decode" else chunk.run
    for part in (0, 128):
        zeros = run(refill(c, hidden, 0.0), part)
        sc.check(c, zeros, "zeros")
        for value in (1.0, 400.0):
            assert torch.equal(run(refill(c, hidden, value), part), zeros), (part, value)


@pytest.mark.parametrize("cap", [0.0, 2.0, 6.0, 40.0])
@pytest.mark.parametrize("kernel", sorted(KERNELS))
@pytest.mark.parametrize("dt,cdt", [("bf16", "bf16"), ("f16", "fp8")])
def test_another_document_does_not_change_a_bit(cap, kernel, dt, cdt):
    """Rows that start at their own document, beside rows of the same tile that see the one
    before: keys of the one before are changed, then grow and shrink."""
    L = KERNELS[kernel][0]
    cached, split = 300, 300 + L // 2
    start = [0] * (L // 2) + [split] * (L - L // 2)
    c = sc.make([cached], [L], 8, 2, 128, 16, dt, cdt, softcap=cap, key_start=start, seed=11)
    before = [(0, t) for t in range(split)]
    for part in (0, 128):
        first = chunk.run(c, part)
        sc.check(c, first, "first")
        for value in (0.01, 5.0, 400.0):
            got = chunk.run(refill(c, before, value), part)
            assert torch.equal(got[L // 2:], first[L // 2:]), (part, value)
            assert not torch.equal(got[:L // 2], first[:L // 2])


@pytest.mark.parametrize("cap", [0.0, 2.0, 6.0, 40.0])
@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_rows_of_the_next_sequence_do_not_change_a_bit(cap, kernel):
    """A query tile's last rows are the next sequence's, which has a tile of its own."""
    L, behind = reversed(KERNELS[kernel])
    c = sc.make([300, 77], [L, behind], 8, 2, 128, 16, "bf16", "bf16", softcap=cap, seed=12)
    for part in (0, 128):
        first = chunk.run(c, part)
        for value in (100.0, float("inf"), float("nan")):
            other = dict(c, q=c["q"].clone())
            other["q"][L:] = value
            assert torch.equal(chunk.run(other, part)[:L], first[:L]), (part, value)
