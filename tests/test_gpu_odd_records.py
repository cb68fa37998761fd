"""Odd numbers of split-K records (sequences x heads x partitions): the rows, read 16 bytes
at a time, stay aligned in every decode that keeps them in a workspace."""
import dataclasses

import pytest
import torch

import paged_kv_cache_338_b200 as pa
import scored_cases as sc
import test_gpu_decode_scored as dec
import test_gpu_shared_prefix as prefix
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pa.pa_device_status(clear=True)
    yield
    pa.pa_decode_select(pa.DECODE_DEFAULT)


def plain(c, partition):
    q = c["q"].cuda()
    S, Hq, D = q.shape
    n = pa.pa_decode_workspace_size(S, Hq, D, c["max_ctx"], partition)
    parts = -(-c["max_ctx"] // partition)
    assert n == S * Hq * parts * (8 + 4 * D) and S * Hq * parts % 2 == 1
    args = (q, c["kc"].cuda(), c["vc"].cuda(), c["tables"].cuda(), c["lens"].cuda(), c["max_ctx"], c["scale"])
    kw = dict(k_scale=c["k_scale"], v_scale=c["v_scale"], partition=partition)
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]
    pa.pa_decode(outs[0], *args, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), **kw)
    pa.pa_decode_noalloc(outs[1], *args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    return outs[0]


@pytest.mark.parametrize("mode", [pa.DECODE_DEFAULT, pa.DECODE_DEFAULT | pa.DECODE_GROUP_PARTITIONS,
                                  pa.DECODE_DEFAULT | pa.DECODE_SIMT_ONLY])
@pytest.mark.parametrize("D,dt,cdt", [(64, "bf16", "bf16"), (128, "f16", "f16"), (128, "bf16", "fp8"),
                                      (256, "bf16", "bf16"), (128, "f32", "f32")])
@pytest.mark.parametrize("S,H", [(1, 1), (3, 3), (5, 1)])
def test_decode(S, H, D, dt, cdt, mode):
    lens = [150, 33, 1, 149, 64][:S]
    c = dec.decode(lens, H, H, D, 16, dt, cdt, seed=S + D)
    want = sc.oracle(c)
    pa.pa_decode_select(mode)
    try:
        for part in (32, 64, 144):               # 5 and 3 partitions, and 2
            if part == 144:
                sc.check(c, dec.run(c, part), "even", want)
                continue
            sc.check(c, plain(c, part), f"pa_decode {part}", want)
            sc.check(c, dec.run(c, part), f"pa_decode_scored {part}", want)
    finally:
        pa.pa_decode_select(pa.DECODE_DEFAULT)
    assert pa.pa_device_status() == 0


@pytest.mark.parametrize("max_ctx", [0, 5128])          # one CTA a suffix; split suffixes
@pytest.mark.parametrize("kv,bs", [("bf16", 16), ("fp8_e4m3", 32)])
def test_shared_prefix(kv, bs, max_ctx):
    base = dataclasses.replace(wl.DECODE_WORKLOADS["prefix_shared_fp8_b256"], kv_dtype=kv, block_size=bs,
                               num_q_heads=3, num_kv_heads=3, fp8_scaled=kv == "fp8_e4m3")
    inp = wl.make_decode_inputs(wl.small_variant(base, 5, 1, 100, prefix_tokens=128), seed=3)
    kc, vc = prefix._appended(inp)
    got = prefix._run(inp, kc, vc, inp.block_tables, inp.context_lens, 128, max(max_ctx, inp.max_ctx))
    prefix._check(got, inp, kc, vc, inp.block_tables, inp.context_lens, kv)
    assert pa.pa_device_status() == 0
