"""Host checks of the fused append and the attentions with modified scores: what
they refuse before anything is enqueued (no GPU), their sizes and splits."""
import ctypes

import pytest

import paged_kv_cache_338_b200 as pa

INVALID, UNSUPPORTED = 1, 2
PTR = 1 << 20                                    # 16-byte aligned, never followed


def call(name, defaults, **kw):
    a = dict(defaults)
    unknown = set(kw) - set(a)
    assert not unknown, unknown
    a.update(kw)
    return getattr(pa.lib(), name)(*a.values())


DECODE = dict(out=PTR, q=PTR, q_dt=2, kc=PTR, vc=PTR, c_dt=2, bt=PTR, MB=4, cl=PTR, S=2, Hq=8,
              Hkv=2, D=128, bs=16, NB=10, max_ctx=64, scale=0.1, ks=1.0, vs=1.0, softcap=0.0,
              slopes=None, window=0, key_start=None, partition=0, ws=None, wsb=0, stream=None)
CHUNK = dict(out=PTR, q=PTR, q_dt=2, kc=PTR, vc=PTR, c_dt=2, bt=PTR, MB=4, cl=PTR, qs=PTR, S=2, T=6,
             Hq=8, Hkv=2, D=128, bs=16, NB=10, max_new=4, max_ctx=640, scale=0.1, ks=1.0, vs=1.0,
             softcap=0.0, slopes=None, window=0, key_start=None, prefix=None, partition=0, ws=None,
             wsb=0, stream=None)
APPEND = dict(qo=PTR, qos=1024, q=PTR, q_s=1024, k=PTR, k_s=256, v=PTR, v_s=256, dt=2, qw=None,
              kw_=None, eps=1e-6, off=0.0, cs=PTR, rows=100, pos=PTR, rot=128, inter=0, kc=PTR,
              vc=PTR, c_dt=2, slots=PTR, T=4, Hq=8, Hkv=2, D=128, bs=16, NB=10, ks=1.0, vs=1.0,
              stream=None)
NAN, INF = float("nan"), float("inf")

SCORE = [(dict(softcap=-1.0), INVALID), (dict(softcap=NAN), INVALID), (dict(softcap=INF), INVALID),
         (dict(softcap=1e-44), INVALID), (dict(window=-1), INVALID), (dict(partition=-128), INVALID),
         (dict(scale=NAN), INVALID), (dict(ks=2.0), INVALID),
         (dict(c_dt=3, ks=0.0), INVALID), (dict(c_dt=3, vs=INF), INVALID), (dict(q_dt=9), INVALID),
         (dict(c_dt=0), UNSUPPORTED), (dict(q_dt=3, c_dt=3), UNSUPPORTED), (dict(Hkv=3), INVALID),
         (dict(Hq=24, Hkv=8), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(bs=64), UNSUPPORTED),
         (dict(S=-1), INVALID), (dict(NB=0), INVALID), (dict(MB=0), INVALID), (dict(q=PTR + 8), INVALID),
         (dict(kc=PTR + 4), INVALID), (dict(bt=None), INVALID), (dict(partition=128), INVALID),
         (dict(partition=128, ws=PTR, wsb=64), INVALID)]


@pytest.mark.parametrize("kw,status", SCORE, ids=lambda x: str(x))
def test_decode_refuses(kw, status):
    assert call("pa_decode_scored", DECODE, **dict(dict(max_ctx=640, MB=40), **kw)) == status
    assert pa.pa_last_error()


@pytest.mark.parametrize("kw,status", SCORE + [
    (dict(D=64, c_dt=3), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(qs=None), INVALID),
    (dict(partition=64), INVALID), (dict(partition=128, ws=PTR + 8, wsb=1 << 30), INVALID),
    (dict(T=-1), INVALID), (dict(max_new=-1), INVALID), (dict(max_ctx=-1), INVALID),
    (dict(scale=-0.1), INVALID), (dict(scale=0.0), INVALID), (dict(S=70000), UNSUPPORTED),
    (dict(softcap=3e38), INVALID), (dict(q_dt=0, c_dt=0), UNSUPPORTED),
    (dict(max_ctx=2 ** 30 + 1), UNSUPPORTED),
], ids=lambda x: str(x))
def test_chunk_refuses(kw, status):
    assert call("pa_prefill_scored", CHUNK, **dict(dict(MB=40), **kw)) == status
    assert pa.pa_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3, c_dt=3), UNSUPPORTED), (dict(dt=2, c_dt=1), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(rot=130), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=-16), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(off=INF), INVALID),
    (dict(q_s=1000), INVALID), (dict(k_s=128), INVALID), (dict(v_s=257), INVALID),
    (dict(q=PTR + 2), INVALID), (dict(cs=None), INVALID), (dict(pos=None), INVALID),
    (dict(rows=0), INVALID), (dict(slots=None), INVALID), (dict(ks=2.0), INVALID),
    (dict(c_dt=3, ks=-1.0), INVALID), (dict(T=-1), INVALID), (dict(NB=1 << 62), INVALID),
    (dict(qw=PTR + 8), INVALID), (dict(cs=PTR + 4), INVALID),
], ids=lambda x: str(x))
def test_append_refuses(kw, status):
    assert call("pa_norm_rope_append", APPEND, **kw) == status
    assert pa.pa_last_error()


def test_nothing_to_do_needs_no_gpu():
    assert call("pa_norm_rope_append", APPEND, T=0) == 0
    assert call("pa_decode_scored", DECODE, S=0) == 0
    for kw in (dict(S=0), dict(T=0), dict(max_new=0)):
        assert call("pa_prefill_scored", CHUNK, **kw) == 0


def test_workspace_sizes():
    f = pa.pa_prefill_scored_workspace_size
    assert f(2, 6, 8, 128, 4, 640, 0, 0) == 0
    assert f(2, 6, 8, 128, 4, 640, 0, 640) == 0
    assert f(2, 6, 8, 128, 4, 640, 0, 128) >= 6 * 8 * 5 * (8 + 512)
    assert f(2, 6, 8, 128, 4, 64000, 100, 128) == 0           # a window fits one part
    assert f(2, 6, 8, 128, 30, 64000, 100, 128) >= 6 * 8 * 2 * (8 + 512)
    assert f(0, 0, 8, 128, 4, 640, 0, 128) == 0
    for bad in ((2, 6, 8, 128, 4, 640, 0, 100), (2, 6, 8, 128, 4, 640, -1, 128),
                (2, -6, 8, 128, 4, 640, 0, 128), (2, 2 ** 31 - 1, 2 ** 30, 2 ** 30, 4, 2 ** 31 - 1, 0, 128)):
        with pytest.raises(pa.PaError):
            f(*bad)
    g = pa.pa_decode_scored_workspace_size
    assert g(3, 8, 128, 16, 1000, 0, 0) == 0
    assert g(3, 8, 128, 16, 1000, 0, 64) == pa.pa_decode_workspace_size(3, 8, 128, 1000, 64)
    assert g(3, 8, 128, 16, 1000, 100, 64) == pa.pa_decode_workspace_size(3, 8, 128, 115, 64)


def test_tiny_batches_split_further():
    f = pa.pa_decode_suggest_partition
    assert f(8, 16, [501]) == 32 and f(8, 16, [200]) == 32
    assert f(1, 16, [1025]) == 64 and f(1, 8, [1024]) == 32   # 32 records a head from 32
    assert f(8, 16, [4000]) == 128                            # 16 x 8 partitions of 256: 128 < 148
    assert f(8, 16, [2000] * 3) == 256                        # 3 x 8 x 8 = 192
    assert f(8, 16, [128]) == 0 and f(8, 16, [200] * 16) == 0 # short ones stay in one pass
    assert f(8, 16, [501] * 64) == 256 and f(32, 16, [64] * 4096) == 0


def test_suggested_parts():
    f = pa.pa_prefill_scored_suggest_partition
    for S in (1, 3, 16, 200):
        for Hq, Hkv in ((8, 8), (32, 8), (16, 1)):
            for L in (0, 1, 8, 300, 5000):
                for n in (0, 1, 500, 40000, 2 ** 31 - 1):
                    for w in (0, 1, 1024):
                        p = f(S, Hq, Hkv, L, n, w)
                        assert p % 128 == 0 and p >= 0
    assert f(64, 32, 8, 2048, 8192, 0) == 0                   # enough CTAs without a split
    assert f(16, 32, 8, 8, 1820, 0) == 0                      # short contexts
    assert 4096 <= f(16, 32, 8, 8, 31969, 0) <= 12288
    assert 512 <= f(1, 32, 8, 8, 9728, 0) <= 1536
    assert f(1, 32, 8, 4, 100000, 0) > 0
    with pytest.raises(pa.PaError):
        f(1, 8, 3, 1, 1, 0)
    with pytest.raises(pa.PaError):
        f(1, 8, 2, -1, 1, 0)
    assert pa.lib().pa_prefill_scored_suggest_partition(1, 8, 2, 1, 1, 0, ctypes.POINTER(ctypes.c_int)()) == INVALID
