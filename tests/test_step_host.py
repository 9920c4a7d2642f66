"""The step operators' host-side checks: every refusal returns its status before any CUDA call (no GPU needed), the
binding refuses tensors it cannot pass on, and the plain references of the GPU tests hold their own definitions."""
import ctypes
import math
import random

import pytest
import torch

import step_reference as R
from paged_attention_decode_gb300 import build as pa_build
from paged_attention_decode_gb300 import pa_v2 as pa

FAKE = 1 << 20          # a non-null, 16-byte aligned address that nothing may touch


@pytest.fixture(scope="module", autouse=True)
def _built():
    pa_build.build()


TABLES = dict(cached=FAKE, new=FAKE, batch=2, table=FAKE, width=4, free=FAKE, num_free=3, parents=FAKE, page_size=16,
              window=0, indptr=FAKE, indices=FAKE, index_capacity=8, lpl=FAKE, fpo=FAKE, qo=FAKE, slots=FAKE,
              positions=FAKE, token_capacity=8, mask=FAKE, mask_words=1, needed=FAKE, status=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(cached=None), pa.PA_EINVAL), (dict(new=None), pa.PA_EINVAL), (dict(batch=-1), pa.PA_EINVAL),
    (dict(table=None), pa.PA_EINVAL), (dict(width=-1), pa.PA_EINVAL), (dict(num_free=-1), pa.PA_EINVAL),
    (dict(page_size=0), pa.PA_EINVAL), (dict(window=-1), pa.PA_EINVAL), (dict(indptr=None), pa.PA_EINVAL),
    (dict(indices=None), pa.PA_EINVAL), (dict(index_capacity=-1), pa.PA_EINVAL), (dict(lpl=None), pa.PA_EINVAL),
    (dict(fpo=None), pa.PA_EINVAL), (dict(qo=None), pa.PA_EINVAL), (dict(slots=None), pa.PA_EINVAL),
    (dict(positions=None), pa.PA_EINVAL), (dict(token_capacity=-1), pa.PA_EINVAL), (dict(mask_words=0), pa.PA_EINVAL),
    (dict(mask_words=-1), pa.PA_EINVAL), (dict(needed=None), pa.PA_EINVAL),
    (dict(batch=pa.MAX_TABLE_BATCH + 1), pa.PA_EUNSUPPORTED), (dict(width=2**30), pa.PA_EUNSUPPORTED),
    (dict(index_capacity=2**31), pa.PA_EUNSUPPORTED), (dict(token_capacity=2**31), pa.PA_EUNSUPPORTED),
    (dict(token_capacity=2**30, mask_words=2), pa.PA_EUNSUPPORTED)])
def test_build_tables_refusals(change, want):
    assert pa.lib().pa_v2_build_tables(*{**TABLES, **change}.values()) == want


QK = dict(q=FAKE, qs=4 * 64, k=FAKE, ks=2 * 64, v=FAKE, vs=2 * 64, dtype=pa.PA_F16, tokens=3, hq=4, hkv=2, D=64,
          pos=FAKE, slots=FAKE, freq=FAKE, rot=64, inter=0, qw=FAKE, kw=FAKE, eps=1e-6, out=FAKE, q_dtype=pa.PA_F16,
          kp=FAKE, vp=FAKE, pages=10, page_size=16, status=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), pa.PA_EINVAL), (dict(k=None), pa.PA_EINVAL), (dict(v=None), pa.PA_EINVAL),
    (dict(pos=None), pa.PA_EINVAL), (dict(slots=None), pa.PA_EINVAL), (dict(freq=None), pa.PA_EINVAL),
    (dict(out=None), pa.PA_EINVAL), (dict(kp=None), pa.PA_EINVAL), (dict(vp=None), pa.PA_EINVAL),
    (dict(tokens=-1), pa.PA_EINVAL), (dict(hq=0), pa.PA_EINVAL), (dict(hkv=0), pa.PA_EINVAL),
    (dict(rot=-16), pa.PA_EINVAL), (dict(pages=0), pa.PA_EINVAL), (dict(page_size=0), pa.PA_EINVAL),
    (dict(eps=-1.0), pa.PA_EINVAL), (dict(eps=math.nan), pa.PA_EINVAL), (dict(eps=math.inf), pa.PA_EINVAL),
    (dict(qs=4 * 64 - 8), pa.PA_EINVAL), (dict(ks=8), pa.PA_EINVAL), (dict(vs=2 * 64 + 4), pa.PA_EINVAL),
    (dict(q=FAKE + 2), pa.PA_EINVAL), (dict(out=FAKE + 8), pa.PA_EINVAL), (dict(kp=FAKE + 4), pa.PA_EINVAL),
    (dict(qw=FAKE + 2), pa.PA_EINVAL), (dict(kw=FAKE + 8), pa.PA_EINVAL),
    (dict(dtype=5), pa.PA_EUNSUPPORTED), (dict(q_dtype=pa.PA_BF16), pa.PA_EUNSUPPORTED),
    (dict(dtype=pa.PA_F32, q_dtype=pa.PA_F16), pa.PA_EUNSUPPORTED), (dict(D=96), pa.PA_EUNSUPPORTED),
    (dict(D=512, qs=2048, ks=1024, vs=1024), pa.PA_EUNSUPPORTED), (dict(rot=24), pa.PA_EUNSUPPORTED),
    (dict(rot=80), pa.PA_EUNSUPPORTED), (dict(pages=2**27), pa.PA_EUNSUPPORTED),
    (dict(pages=2**40), pa.PA_EUNSUPPORTED)])
def test_qk_rope_append_refusals(change, want):
    assert pa.lib().pa_v2_qk_rope_append(*{**QK, **change}.values()) == want


def test_qk_rope_append_without_tokens_does_nothing():
    assert pa.lib().pa_v2_qk_rope_append(*{**QK, "tokens": 0}.values()) == pa.PA_OK


TREE = dict(q=FAKE, kp=FAKE, vp=FAKE, dtype=pa.PA_BF16, pages=10, page_size=16, hq=8, hkv=2, D=128, idx=FAKE, n_idx=5,
            indptr=FAKE, lpl=FAKE, fpo=FAKE, batch=2, qo=FAKE, tokens=7, mask=FAKE, words=1, scale=0.1, out=FAKE,
            lse=FAKE, ws=FAKE, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), pa.PA_EINVAL), (dict(kp=None), pa.PA_EINVAL), (dict(vp=None), pa.PA_EINVAL),
    (dict(idx=None), pa.PA_EINVAL), (dict(indptr=None), pa.PA_EINVAL), (dict(lpl=None), pa.PA_EINVAL),
    (dict(fpo=None), pa.PA_EINVAL), (dict(qo=None), pa.PA_EINVAL), (dict(out=None), pa.PA_EINVAL),
    (dict(lse=None), pa.PA_EINVAL), (dict(ws=None), pa.PA_EINVAL), (dict(pages=0), pa.PA_EINVAL),
    (dict(page_size=0), pa.PA_EINVAL), (dict(hq=0), pa.PA_EINVAL), (dict(hkv=0), pa.PA_EINVAL),
    (dict(hq=7), pa.PA_EINVAL), (dict(hq=1), pa.PA_EINVAL), (dict(batch=-1), pa.PA_EINVAL),
    (dict(tokens=-1), pa.PA_EINVAL), (dict(n_idx=-1), pa.PA_EINVAL), (dict(words=0), pa.PA_EINVAL),
    (dict(words=-1, mask=None), pa.PA_EINVAL), (dict(scale=math.nan), pa.PA_EINVAL),
    (dict(scale=math.inf), pa.PA_EINVAL), (dict(q=FAKE + 2), pa.PA_EINVAL), (dict(kp=FAKE + 8), pa.PA_EINVAL),
    (dict(vp=FAKE + 2), pa.PA_EINVAL), (dict(out=FAKE + 2), pa.PA_EINVAL), (dict(ws=FAKE + 4), pa.PA_EINVAL),
    (dict(dtype=pa.PA_F32), pa.PA_EUNSUPPORTED), (dict(dtype=9), pa.PA_EUNSUPPORTED), (dict(D=96), pa.PA_EUNSUPPORTED),
    (dict(D=512), pa.PA_EUNSUPPORTED), (dict(page_size=17), pa.PA_EUNSUPPORTED), (dict(page_size=272), pa.PA_EUNSUPPORTED),
    (dict(pages=2**27), pa.PA_EUNSUPPORTED), (dict(words=pa.MAX_MASK_WORDS + 1), pa.PA_EUNSUPPORTED)])
def test_tree_attention_refusals(change, want):
    assert pa.lib().pa_v2_tree_attention(*{**TREE, **change}.values()) == want


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_tree_attention_refuses_scales_that_overflow_in_base_2(scale):
    assert pa.lib().pa_v2_tree_attention(*{**TREE, "scale": scale}.values()) == pa.PA_EUNSUPPORTED


def test_tree_attention_without_work_does_nothing():
    for change in (dict(tokens=0), dict(batch=0)):
        assert pa.lib().pa_v2_tree_attention(*{**TREE, **change}.values()) == pa.PA_OK


SLIDING = {k: v for key, value in TREE.items() for k, v in
           ((("positions", FAKE), ("window", 64), (key, value)) if key == "scale" else ((key, value),))}


@pytest.mark.parametrize("change,want", [
    (dict(window=0), pa.PA_EINVAL), (dict(window=-1), pa.PA_EINVAL), (dict(positions=None), pa.PA_EINVAL),
    (dict(q=None), pa.PA_EINVAL), (dict(words=0), pa.PA_EINVAL), (dict(scale=math.nan), pa.PA_EINVAL),
    (dict(hq=7), pa.PA_EINVAL), (dict(dtype=pa.PA_F32), pa.PA_EUNSUPPORTED), (dict(D=96), pa.PA_EUNSUPPORTED),
    (dict(words=pa.MAX_MASK_WORDS + 1), pa.PA_EUNSUPPORTED)])
def test_tree_attention_sliding_refusals(change, want):
    assert list(SLIDING)[17:22] == ["mask", "words", "positions", "window", "scale"]
    assert pa.lib().pa_v2_tree_attention_sliding(*{**SLIDING, **change}.values()) == want


def test_tree_attention_sliding_without_work_does_nothing():
    for change in (dict(tokens=0), dict(batch=0)):
        assert pa.lib().pa_v2_tree_attention_sliding(*{**SLIDING, **change}.values()) == pa.PA_OK


@pytest.mark.parametrize("change,want", [
    (dict(window=0), pa.PA_EINVAL), (dict(window=-1), pa.PA_EINVAL), (dict(cached=None), pa.PA_EINVAL),
    (dict(page_size=0), pa.PA_EINVAL), (dict(mask_words=0), pa.PA_EINVAL),
    (dict(batch=pa.MAX_TABLE_BATCH + 1), pa.PA_EUNSUPPORTED)])
def test_build_tables_sliding_refusals(change, want):
    assert pa.lib().pa_v2_build_tables_sliding(*{**TABLES, "window": 5, **change}.values()) == want


def test_binding_refuses_two_windows():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="not both"):
        pa.pa_v2_build_tables(z, z, torch.zeros(4, 4, dtype=torch.int32), 16, pa.StepTables.empty(4, 8, 8, 1, device="cpu"),
                              window=3, sliding_window=3)


def test_tree_attention_workspace_refusals():
    n = ctypes.c_int64()
    f = pa.lib().pa_v2_tree_attention_workspace
    assert f(0, 4, 2, 8, 2, 128, None) == pa.PA_EINVAL
    for bad in ((-1, 4, 2, 8, 2, 128), (0, -4, 2, 8, 2, 128), (0, 4, -2, 8, 2, 128), (0, 4, 2, 7, 2, 128), (0, 4, 2, 8, 0, 128)):
        assert f(*bad, ctypes.byref(n)) == pa.PA_EINVAL, bad
    assert f(0, 4, 2, 8, 2, 96, ctypes.byref(n)) == pa.PA_EUNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_shapes():
    z = torch.zeros(4, dtype=torch.int32)
    t = pa.StepTables.empty(4, 8, 8, 1, device="cpu")
    with pytest.raises(ValueError):
        pa.pa_v2_build_tables(z, z, torch.zeros(4, 4, dtype=torch.int32), 16, t)
    with pytest.raises(ValueError):
        pa.pa_v2_build_tables(z, z, z, 16, t)
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    pool = torch.zeros(3, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.pa_v2_qk_rope_append(x, x, x, z, z, None, pool, pool)
    with pytest.raises(ValueError):
        pa.pa_v2_tree_attention(x, pool, pool, z, z, z, z, z, 0.1)
    with pytest.raises(ValueError):
        pa.pa_v2_tree_attention(x, pool, pool.float(), z, z, z, z, z, 0.1)


# ---------------------------------------------------------------------------
# the references themselves
# ---------------------------------------------------------------------------

def test_reference_tables_of_a_worked_example():
    # 4-entry pages; request 0: 5 cached + 4 new with tree -1,0,0,1; request 1: 8 cached (two full pages) + 1
    table = torch.tensor([[3, 9, -1, -1], [5, 6, -1, -1]], dtype=torch.int32)
    ref = R.tables_ref([5, 8], [4, 1], table, torch.tensor([20, 21, 22]), [[-1, 0, 0, 1], [-1]], 4, 6, 1)
    assert ref["block_table"].tolist() == [[3, 9, 20, -1], [5, 6, 21, -1]] and ref["pages_needed"] == 2
    assert ref["indices"] == [3, 9, 20, 5, 6, 21] and ref["indptr"] == [0, 3, 6]     # both windows start at token 3
    assert ref["first_page_offset"] == [3, 3] and ref["last_page_len"] == [1, 1]
    assert ref["slots"] == [9 * 4 + 1, 9 * 4 + 2, 9 * 4 + 3, 20 * 4, 21 * 4]
    assert ref["positions"] == [5, 6, 6, 7, 8]
    assert ref["tree_mask"] == [[1], [3], [5], [11], [1]]


def test_reference_mask_words_hold_every_bit():
    parents = list(range(-1, 69))
    m = R.tree_mask([parents], 3)
    assert m[31].tolist() == [-1, 0, 0] and m[63].tolist() == [-1, -1, 0] and m[64].tolist() == [-1, -1, 1]


def test_reference_rotation_turns_pairs():
    x = torch.zeros(1, 1, 64)
    x[0, 0, 0] = 1.0
    half, _ = R.rope_ref(x, None, 0.0, [1], [math.pi / 2] * 32, False)
    assert abs(float(half[0, 0, 32]) - 1) < 1e-7 and abs(float(half[0, 0, 0])) < 1e-7
    inter, _ = R.rope_ref(x, None, 0.0, [1], [math.pi / 2] * 32, True)
    assert abs(float(inter[0, 0, 1]) - 1) < 1e-7
    rms, _ = R.rope_ref(torch.full((1, 1, 64), 3.0), torch.full((64,), 2.0), 0.0, [0], [], False)
    assert torch.allclose(rms, torch.full((1, 1, 64), 2.0, dtype=torch.float64))


def test_reference_attention_equals_dense_softmax():
    rng = random.Random(1)
    g = torch.Generator().manual_seed(1)
    q, kp, vp = torch.randn(5, 2, 64, generator=g), torch.randn(9, 4, 1, 64, generator=g), torch.randn(9, 4, 1, 64, generator=g)
    tree = R.random_tree(rng, 5, 0.0)
    idx = torch.tensor([7, 2, 5], dtype=torch.int32)
    ro, rl, _, _ = R.attention_ref(q.half(), kp.half(), vp.half(), idx, [0, 3], [3], [1], [0, 5], 0.125,
                                   R.tree_mask([tree], 1))
    rows = torch.cat([torch.arange(4) + 4 * p for p in (7, 2, 5)])[1:11]
    k, v = kp.half().double().flatten(0, 1)[rows, 0], vp.half().double().flatten(0, 1)[rows, 0]
    allow = torch.ones(5, 10, dtype=torch.bool)
    for i in range(5):
        for j in range(5):
            allow[i, 5 + j] = j in R.ancestors(tree, i)
    for h in range(2):
        o = torch.nn.functional.scaled_dot_product_attention(q.half().double()[None, :, h], k[None], v[None], attn_mask=allow,
                                                             scale=0.125)[0]
        assert (o - ro[:, h]).abs().max() < 1e-12


def test_reference_sliding_tables_of_a_worked_example():
    # window 3, 4-entry pages: a tree behind 9 cached tokens (its roots see tokens 7 and 8), a chain behind 2, no token
    table = torch.tensor([[3, 9, 4, 8], [5, 6, 0, 0], [7, 1, 2, 0]], dtype=torch.int32)
    ref = R.sliding_tables_ref([9, 2, 10], [5, 5, 0], table, None, [[-1, 0, 1, 2, 0], [-1, 0, 1, 2, 3], []], 4, 3, 1)
    assert ref["first_page_offset"] == [3, 0, 3] and ref["last_page_len"] == [2, 3, 2]
    assert ref["indices"] == [9, 4, 8, 5, 6, 1, 2] and ref["indptr"] == [0, 3, 5, 7]
    assert ref["positions"] == [9, 10, 11, 12, 10, 2, 3, 4, 5, 6]
    assert ref["tree_mask"] == [[1], [3], [7], [14], [17], [1], [3], [7], [14], [28]]


def test_reference_rows_attention_equals_the_paged_one():
    g = torch.Generator().manual_seed(3)
    q, kp, vp = (torch.randn(*s, generator=g).half() for s in ((2, 4, 64), (5, 4, 2, 64), (5, 4, 2, 64)))
    idx = torch.tensor([3, 1], dtype=torch.int32)
    paged = R.attention_ref(q, kp, vp, idx, [0, 2], [3], [1], [0, 2], 0.1)
    rows = [13, 14, 15, 4, 5, 6]
    alone = R.rows_attention_ref(q, kp, vp, [rows[:5], rows], 0.1)
    assert all(torch.allclose(a, b, atol=1e-13) for a, b in zip(paged, alone))
