"""The 8-bit cache's host-side checks: every refusal returns its status before any CUDA call (no GPU needed), the
binding refuses tensors that it cannot pass on, and the plain references hold their own definitions."""
import ctypes
import math

import pytest
import torch

import fp8_reference as F
from paged_attention_decode_gb300 import build as pa_build
from paged_attention_decode_gb300 import pa_v2 as pa

FAKE = 1 << 20          # a non-null, 16-byte aligned address that nothing may touch


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa_build.build()


APPEND = dict(q=FAKE, qs=4 * 64, k=FAKE, ks=2 * 64, v=FAKE, vs=2 * 64, dtype=pa.PA_F16, tokens=3, hq=4, hkv=2, D=64,
              pos=FAKE, slots=FAKE, freq=FAKE, rot=64, inter=0, qw=FAKE, kw=FAKE, eps=1e-6, out=FAKE,
              q_dtype=pa.PA_F16, kp=FAKE, vp=FAKE, ke=FAKE, ve=FAKE, pages=10, page_size=16, status=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), pa.PA_EINVAL), (dict(k=None), pa.PA_EINVAL), (dict(v=None), pa.PA_EINVAL),
    (dict(pos=None), pa.PA_EINVAL), (dict(slots=None), pa.PA_EINVAL), (dict(freq=None), pa.PA_EINVAL),
    (dict(out=None), pa.PA_EINVAL), (dict(kp=None), pa.PA_EINVAL), (dict(vp=None), pa.PA_EINVAL),
    (dict(ke=None), pa.PA_EINVAL), (dict(ve=None), pa.PA_EINVAL), (dict(tokens=-1), pa.PA_EINVAL),
    (dict(hq=0), pa.PA_EINVAL), (dict(hkv=0), pa.PA_EINVAL), (dict(rot=-16), pa.PA_EINVAL),
    (dict(pages=0), pa.PA_EINVAL), (dict(page_size=0), pa.PA_EINVAL), (dict(eps=-1.0), pa.PA_EINVAL),
    (dict(eps=math.nan), pa.PA_EINVAL), (dict(qs=4 * 64 - 8), pa.PA_EINVAL), (dict(ks=8), pa.PA_EINVAL),
    (dict(vs=2 * 64 + 4), pa.PA_EINVAL), (dict(q=FAKE + 2), pa.PA_EINVAL), (dict(out=FAKE + 8), pa.PA_EINVAL),
    (dict(kp=FAKE + 4), pa.PA_EINVAL), (dict(kw=FAKE + 8), pa.PA_EINVAL),
    (dict(dtype=pa.PA_E4M3), pa.PA_EUNSUPPORTED), (dict(q_dtype=pa.PA_BF16), pa.PA_EUNSUPPORTED),
    (dict(dtype=pa.PA_F32, q_dtype=pa.PA_F16), pa.PA_EUNSUPPORTED), (dict(D=96), pa.PA_EUNSUPPORTED),
    (dict(rot=24), pa.PA_EUNSUPPORTED), (dict(rot=80), pa.PA_EUNSUPPORTED), (dict(page_size=257), pa.PA_EUNSUPPORTED),
    (dict(pages=2**27), pa.PA_EUNSUPPORTED), (dict(hq=16385, qs=2**21), pa.PA_EUNSUPPORTED),
    (dict(qs=2**31), pa.PA_EUNSUPPORTED)])
def test_append_refusals(change, want):
    assert pa.lib().pa_v2_qk_rope_append_fp8(*{**APPEND, **change}.values()) == want


def test_append_without_tokens_does_nothing():
    assert pa.lib().pa_v2_qk_rope_append_fp8(*{**APPEND, "tokens": 0}.values()) == pa.PA_OK


ATTN = dict(q=FAKE, q_dtype=pa.PA_BF16, kp=FAKE, vp=FAKE, ke=FAKE, ve=FAKE, pages=10, page_size=16, hq=8, hkv=2, D=128,
            idx=FAKE, n_idx=5, indptr=FAKE, lpl=FAKE, fpo=FAKE, batch=2, qo=FAKE, tokens=7, mask=FAKE, words=1,
            pos=FAKE, window=8, sinks=2, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, status=None,
            stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), pa.PA_EINVAL), (dict(kp=None), pa.PA_EINVAL), (dict(vp=None), pa.PA_EINVAL),
    (dict(ke=None), pa.PA_EINVAL), (dict(ve=None), pa.PA_EINVAL), (dict(idx=None), pa.PA_EINVAL),
    (dict(indptr=None), pa.PA_EINVAL), (dict(lpl=None), pa.PA_EINVAL), (dict(fpo=None), pa.PA_EINVAL),
    (dict(qo=None), pa.PA_EINVAL), (dict(out=None), pa.PA_EINVAL), (dict(lse=None), pa.PA_EINVAL),
    (dict(ws=None), pa.PA_EINVAL), (dict(pos=None), pa.PA_EINVAL), (dict(pages=0), pa.PA_EINVAL),
    (dict(page_size=0), pa.PA_EINVAL), (dict(hq=0), pa.PA_EINVAL), (dict(hkv=0), pa.PA_EINVAL),
    (dict(hq=9), pa.PA_EINVAL), (dict(batch=-1), pa.PA_EINVAL), (dict(tokens=-1), pa.PA_EINVAL),
    (dict(n_idx=-1), pa.PA_EINVAL), (dict(words=0), pa.PA_EINVAL), (dict(words=-1), pa.PA_EINVAL),
    (dict(window=-1), pa.PA_EINVAL), (dict(sinks=-1), pa.PA_EINVAL), (dict(window=0), pa.PA_EINVAL),
    (dict(scale=math.inf), pa.PA_EINVAL), (dict(scale=math.nan), pa.PA_EINVAL), (dict(q=FAKE + 2), pa.PA_EINVAL),
    (dict(kp=FAKE + 8), pa.PA_EINVAL), (dict(out=FAKE + 4), pa.PA_EINVAL), (dict(ws=FAKE + 8), pa.PA_EINVAL),
    (dict(q_dtype=pa.PA_F32), pa.PA_EUNSUPPORTED), (dict(q_dtype=pa.PA_E4M3), pa.PA_EUNSUPPORTED),
    (dict(D=96), pa.PA_EUNSUPPORTED), (dict(page_size=17), pa.PA_EUNSUPPORTED),
    (dict(page_size=272), pa.PA_EUNSUPPORTED), (dict(pages=2**27), pa.PA_EUNSUPPORTED),
    (dict(words=33), pa.PA_EUNSUPPORTED), (dict(batch=2**20 + 1), pa.PA_EUNSUPPORTED),
    (dict(scale=3e38), pa.PA_EUNSUPPORTED), (dict(tokens=2**30), pa.PA_EUNSUPPORTED)])
def test_attention_refusals(change, want):
    assert pa.lib().pa_v2_attention_fp8(*{**ATTN, **change}.values()) == want


def test_attention_without_tokens_or_requests_does_nothing():
    assert pa.lib().pa_v2_attention_fp8(*{**ATTN, "tokens": 0}.values()) == pa.PA_OK
    assert pa.lib().pa_v2_attention_fp8(*{**ATTN, "batch": 0}.values()) == pa.PA_OK


@pytest.mark.parametrize("change,want", [
    (dict(device=-1), pa.PA_EINVAL), (dict(tokens=-1), pa.PA_EINVAL), (dict(batch=-1), pa.PA_EINVAL),
    (dict(hkv=0), pa.PA_EINVAL), (dict(hq=7), pa.PA_EINVAL), (dict(D=32), pa.PA_EUNSUPPORTED)])
def test_workspace_refusals(change, want):
    args = {**dict(device=0, tokens=1, batch=1, hq=8, hkv=2, D=128), **change}
    assert pa.lib().pa_v2_attention_fp8_workspace(*args.values(), ctypes.byref(ctypes.c_int64())) == want
    assert pa.lib().pa_v2_attention_fp8_workspace(0, 1, 1, 8, 2, 128, None) == pa.PA_EINVAL


def test_binding_refuses_pools_and_exponents_that_do_not_fit():
    kp = torch.zeros(3, 4, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    ke = torch.zeros(3, 2, dtype=torch.int8)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        pa._pools_fp8(kp.view(torch.uint8), kp, ke, ke, 0)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        pa._pools_fp8(kp, kp[:2], ke, ke, 0)
    with pytest.raises(ValueError, match="num_pages, num_kv_heads"):
        pa._pools_fp8(kp, kp, ke[:2], ke, 0)
    with pytest.raises(ValueError, match="must be \\[num_pages"):
        pa._pools_fp8(kp[0], kp[0], ke, ke, 0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_v2_attention_fp8(torch.zeros(1, 2, 64).half(), kp, kp, ke, ke, None, None, None, None, None, 1.0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_v2_qk_rope_append_fp8(torch.zeros(1, 2, 64).half(), None, None, None, None, None, kp, kp, ke, ke)


def test_reference_codes_are_torchs():
    x = torch.cat([torch.linspace(-460, 460, 4001), torch.randn(4000, generator=torch.Generator().manual_seed(1)),
                   torch.exp2(torch.arange(-13.0, 9)), 3 * torch.exp2(torch.arange(-12.0, 7))]).clamp(-448, 448)
    assert torch.equal(F.code_of(x.double()), x.to(F.E4M3).float().double())
    every = torch.arange(256, dtype=torch.uint8).view(F.E4M3).float()
    fine = every[every.isfinite()].double()
    assert torch.equal(F.code_of(fine), fine) and len(fine) == 254


def test_reference_exponents_hold_the_largest_value():
    for top in (0.0, 1e-9, 448 * 2.0 ** -15, 448 * 2.0 ** -15 * 1.0001, 1.0, 3.5, 3.5001, 448.0, 449.0, 57344.0, 1e9):
        e = F.need_of(top)
        assert F.EXP_MIN <= e <= F.EXP_MAX
        assert e == F.EXP_MAX or top <= 448 * 2.0 ** e
        assert e == F.EXP_MIN or top > 448 * 2.0 ** (e - 1)


def test_every_code_and_exponent_is_a_half():
    codes = torch.arange(256, dtype=torch.uint8).view(F.E4M3).reshape(1, 4, 1, 64).expand(23, 4, 1, 64)
    F.values(codes, torch.arange(-15, 8, dtype=torch.int8).reshape(23, 1))       # asserts it


def test_reference_rows_seen():
    ids, see = [7, 3, 5], F.seen_rows
    assert see(ids, 4, 0, 10, 1, 0) == [28, 29, 30, 31, 12, 13, 14, 15, 20, 21]
    assert see(ids, 4, 0, 10, 1, 0, window=3, sinks=2) == [28, 29, 15, 20, 21]
    assert see(ids, 4, 1, 9, 2, 0, window=3) == [14, 15, 20]
    assert see(ids, 4, 0, 10, 3, 2, window=9, sinks=0, line=[0, 2], depth=1) == [28, 29, 30, 31, 12, 13, 14, 15, 21]
