"""Attention with a window and sinks: host-side refusals (no GPU needed)."""
import math

import pytest
import torch

from paged_attention_decode_gb300 import build as pa_build
from paged_attention_decode_gb300 import pa_v2 as pa

FAKE = 1 << 20          # a non-null, 16-byte aligned address that nothing may touch


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa_build.build()


SINKS = dict(q=FAKE, kp=FAKE, vp=FAKE, dtype=pa.PA_BF16, pages=10, page_size=16, hq=8, hkv=2, D=128, idx=FAKE, n_idx=5,
             indptr=FAKE, lpl=FAKE, fpo=FAKE, batch=2, qo=FAKE, tokens=7, mask=FAKE, words=1, positions=FAKE, window=9,
             sinks=4, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(window=0), pa.PA_EINVAL), (dict(window=-1), pa.PA_EINVAL), (dict(sinks=0), pa.PA_EINVAL),
    (dict(sinks=-1), pa.PA_EINVAL), (dict(positions=None), pa.PA_EINVAL), (dict(q=None), pa.PA_EINVAL),
    (dict(words=0), pa.PA_EINVAL), (dict(scale=math.nan), pa.PA_EINVAL), (dict(hq=7), pa.PA_EINVAL),
    (dict(kp=FAKE + 8), pa.PA_EINVAL), (dict(dtype=pa.PA_F32), pa.PA_EUNSUPPORTED),
    (dict(dtype=pa.PA_E4M3), pa.PA_EUNSUPPORTED), (dict(D=96), pa.PA_EUNSUPPORTED),
    (dict(page_size=20), pa.PA_EUNSUPPORTED), (dict(words=pa.MAX_MASK_WORDS + 1), pa.PA_EUNSUPPORTED)])
def test_tree_attention_sinks_refusals(change, want):
    assert pa.lib().pa_v2_tree_attention_sinks(*{**SINKS, **change}.values()) == want


def test_tree_attention_sinks_without_work_does_nothing():
    for change in (dict(tokens=0), dict(batch=0)):
        assert pa.lib().pa_v2_tree_attention_sinks(*{**SINKS, **change}.values()) == pa.PA_OK


def test_an_8_bit_cache_is_no_kv_dtype_of_the_other_calls():
    z = torch.zeros(2, 4, 1, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pa._pools(z, z, 0)
    assert pa.pa_v2_q_heads_per_cta(4, 128, pa.PA_E4M3) == 0
