"""Factors that the modified-score attentions refuse on the host (no GPU)."""
import pytest

import paged_kv_cache_338_b200 as pa
from test_scored_host import CHUNK, DECODE, INVALID, call


@pytest.mark.parametrize("kw", [dict(softcap=1.7e38, scale=0.0884), dict(softcap=1e30, scale=1e-10),
                                dict(softcap=1e20, scale=-1e-20)])
def test_caps_that_leave_no_normal_factor(kw):
    assert call("pa_decode_scored", DECODE, **kw) == INVALID
    assert "softcap" in pa.pa_last_error()
    assert call("pa_prefill_scored", CHUNK, **dict(dict(MB=40), **kw)) == INVALID
