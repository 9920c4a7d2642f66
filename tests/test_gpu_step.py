"""GPU: the step operators (pa_v2_build_tables, pa_v2_qk_rope_append, pa_v2_tree_attention) against plain 64-bit
references, alone and together."""
import math
import random

import pytest
import torch

import step_reference as R
from paged_attention_decode_gb300 import pa_v2 as pa

pytestmark = pytest.mark.gpu

I32 = torch.int32
FIELDS = ("indptr", "indices", "last_page_len", "first_page_offset", "qo_indptr", "slots", "positions", "tree_mask",
          "pages_needed")


def i32(x):
    return torch.tensor(list(x), dtype=I32)


def status_word():
    return torch.zeros(1, dtype=I32, device="cuda")


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def _fresh_tables(B, cap_i, cap_t, words):
    t = pa.StepTables.empty(B, cap_i, cap_t, words)
    for f in FIELDS:
        x = getattr(t, f)
        if x is not None:
            x.fill_(-77)
    return t


def _tables_case(seed, B, page_size, ctx, new, tree, window, free_list, spare):
    rng = random.Random(seed)
    cached = [rng.choice([0, 1, page_size - 1, page_size, rng.randint(0, ctx)]) for _ in range(B)]
    fresh = [rng.choice([0, 1, new, rng.randint(0, new)]) for _ in range(B)]
    parents = [R.random_tree(rng, n) for n in fresh] if tree else None
    width = max(1, max(-(-(c + n) // page_size) for c, n in zip(cached, fresh)) + rng.randint(0, 3))
    taken = sum(-(-(c + n) // page_size) - -(-c // page_size) for c, n in zip(cached, fresh))
    ids = torch.randperm(B * width + taken + 5, generator=torch.Generator().manual_seed(seed)).to(I32)
    table, free = ids[:B * width].reshape(B, width).clone(), ids[B * width:].clone()
    cap_i = sum(-(-(c + n) // page_size) for c, n in zip(cached, fresh)) + rng.choice([0, 9])
    cap_t = sum(fresh) + spare
    words = -(-max(max(fresh), 1) // 32) if tree else 0
    return cached, fresh, parents, table, (free if free_list else None), cap_i, cap_t, words


def _run_tables(cached, fresh, parents, table, free, cap_i, cap_t, words, page_size, window, t=None, status=None,
                stream=None):
    B = len(cached)
    t = t if t is not None else _fresh_tables(B, cap_i, cap_t, words)
    packed = None
    if parents is not None:
        flat = [p for ps in parents for p in ps]
        packed = i32(flat + [-1] * (cap_t - len(flat))).cuda()
    dtab = table.cuda()
    pa.pa_v2_build_tables(i32(cached).cuda(), i32(fresh).cuda(), dtab, page_size, t,
                          free_pages=free.cuda() if free is not None else None, parents=packed, window=window,
                          status=status, stream=stream)
    return t, dtab


def _check_tables(t, dtab, ref, cap_t):
    torch.cuda.synchronize()
    assert torch.equal(dtab.cpu(), ref["block_table"])
    for f in ("indptr", "last_page_len", "first_page_offset", "qo_indptr"):
        assert getattr(t, f).tolist() == ref[f], f
    assert int(t.pages_needed) == ref["pages_needed"]
    n, m = len(ref["indices"]), len(ref["slots"])
    assert t.indices[:n].tolist() == ref["indices"]
    assert t.indices[n:].eq(-77).all()
    assert t.slots.tolist() == ref["slots"] + [-1] * (cap_t - m)
    assert t.positions.tolist() == ref["positions"] + [0] * (cap_t - m)
    if t.tree_mask is not None and t.tree_mask.numel():
        assert t.tree_mask[:m].tolist() == ref["tree_mask"]
        assert t.tree_mask[m:].eq(-77).all()


@pytest.mark.parametrize("free_list", [True, False])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B,page_size,ctx,new,window,spare", [
    (1, 16, 0, 1, 0, 0), (1, 16, 5000, 1, 0, 3), (3, 1, 40, 5, 7, 0), (5, 5, 300, 33, 0, 11), (7, 16, 4000, 64, 1024, 0),
    (64, 16, 200, 8, 0, 40), (9, 64, 9000, 70, 4096, 1), (700, 16, 60, 3, 0, 5), (2, 256, 70000, 200, 0, 0)])
def test_tables_match_the_definition(B, page_size, ctx, new, window, spare, tree, free_list):
    case = _tables_case(B * 31 + page_size, B, page_size, ctx, new, tree, window, free_list, spare)
    st = status_word()
    t, dtab = _run_tables(*case, page_size, window, status=st)
    cached, fresh, parents, table, free, _, cap_t, words = case
    ref = R.tables_ref(cached, fresh, table, free, parents, page_size, window, words)
    _check_tables(t, dtab, ref, cap_t)
    assert int(st) == 0


def test_tables_of_a_long_chain_and_chain_masks():
    # a chain without parents still gets its masks when asked for, and positions by index
    t = _fresh_tables(2, 20, 70, 2)
    table = torch.arange(40, dtype=I32).reshape(2, 20)
    pa.pa_v2_build_tables(i32([5, 0]).cuda(), i32([3, 40]).cuda(), table.cuda(), 4, t)
    ref = R.tables_ref([5, 0], [3, 40], table, None, None, 4, 0, 2)
    _check_tables(t, table.cuda(), ref, 70)


def test_tables_window_shorter_than_the_new_tokens():
    """More new tokens than the window: all of them are listed, so that the attention has a row for each; the request
    beside them is cut to the window as ever."""
    ps, cached, fresh, window = 4, [9, 30, 0], [6, 2, 5], 3
    table = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:30].reshape(3, 10).to(I32)
    t, st = _fresh_tables(3, 30, 13, 1), status_word()
    pa.pa_v2_build_tables(i32(cached).cuda(), i32(fresh).cuda(), table.cuda(), ps, t, window=window, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert t.first_page_offset.tolist() == [1, 1, 0] and t.last_page_len.tolist() == [3, 4, 1]   # tokens 9, 29 and 0
    assert t.indptr.tolist() == [0, 2, 3, 5] and t.indices[:5].tolist() == [*table[0, 2:4], table[1, 7], *table[2, :2]]
    # the attention over these tables: 6, 3 and 5 visible tokens, nothing refused
    g = torch.Generator().manual_seed(2)
    kp, vp = (torch.randn(40, ps, 2, 64, generator=g).half() for _ in range(2))
    q = torch.randn(13, 4, 64, generator=g).half()
    out, lse = pa.pa_v2_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), t.indices, t.indptr, t.last_page_len,
                                       t.first_page_offset, t.qo_indptr, 0.125, tree_mask=t.tree_mask, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    ro, rl, to, tl = R.attention_ref(q, kp, vp, t.indices.cpu(), t.indptr.cpu(), t.last_page_len.cpu(),
                                     t.first_page_offset.cpu(), t.qo_indptr.cpu(), 0.125, t.tree_mask.cpu())
    assert ((out.cpu().double() - ro).abs() <= to).all() and ((lse.cpu().double() - rl).abs() <= tl).all()


def test_tables_same_call_again_and_reuse_for_another_batch():
    case = _tables_case(5, 6, 16, 500, 20, True, 0, True, 4)
    cached, fresh, parents, table, free, cap_i, cap_t, words = case
    ref = R.tables_ref(cached, fresh, table, free, parents, 16, 0, words)
    t, dtab = _run_tables(*case, 16, 0)
    _check_tables(t, dtab, ref, cap_t)
    t, dtab = _run_tables(cached, fresh, parents, dtab.cpu(), free, cap_i, cap_t, words, 16, 0, t=t)
    _check_tables(t, dtab, ref, cap_t)


def test_tables_empty_batches():
    t = _fresh_tables(0, 4, 3, 0)
    pa.pa_v2_build_tables(i32([]).cuda(), i32([]).cuda(), torch.zeros(0, 5, dtype=I32, device="cuda"), 16, t)
    assert t.indptr.tolist() == [0] and t.qo_indptr.tolist() == [0] and int(t.pages_needed) == 0
    assert t.slots.tolist() == [-1] * 3 and t.indices.tolist() == [-77] * 4


def test_tables_bad_data_is_contained_and_reported():
    B, ps, width = 5, 4, 3
    table = torch.arange(B * width, dtype=I32).reshape(B, width)
    cached, fresh = [4, -2, 3, 10, 1], [2, 3, -1, 5, 1]      # 1: negative, 2: negative, 3: needs 4 pages
    st = status_word()
    t = _fresh_tables(B, 16, 16, 0)
    d = table.cuda()
    pa.pa_v2_build_tables(i32(cached).cuda(), i32(fresh).cuda(), d, ps, t, status=st)
    torch.cuda.synchronize()
    assert int(st) & pa.DEVICE_BAD_LENGTH
    assert t.indptr.tolist() == [0, 2, 2, 2, 2, 3]
    assert t.indices[:3].tolist() == [0, 1, 12]
    assert t.qo_indptr.tolist() == [0, 2, 5, 5, 10, 11]
    assert t.slots[:11].tolist() == [1 * 4 + 0, 1 * 4 + 1] + [-1] * 8 + [12 * 4 + 1]
    assert t.last_page_len.tolist() == [2, 0, 0, 0, 2]
    assert torch.equal(d.cpu(), table)


def test_tables_short_free_list_and_capacities():
    table = torch.full((2, 4), 50, dtype=I32)
    st = status_word()
    t = _fresh_tables(2, 8, 8, 0)
    d = table.cuda()
    pa.pa_v2_build_tables(i32([0, 0]).cuda(), i32([3, 3]).cuda(), d, 2, t, free_pages=i32([7, 8, 9]).cuda(), status=st)
    torch.cuda.synchronize()
    assert int(st) & pa.DEVICE_NO_PAGES and int(t.pages_needed) == 4
    assert d.tolist() == [[7, 8, 50, 50], [9, -1, 50, 50]]
    assert t.slots[:6].tolist() == [14, 15, 16, 18, 19, -1]
    # index and token capacities: nothing past them is written
    st.zero_()
    t = _fresh_tables(2, 3, 4, 0)
    guard_i, guard_t = torch.full((8,), -77, dtype=I32, device="cuda"), torch.full((8,), -77, dtype=I32, device="cuda")
    t.indices, t.slots = guard_i[:3], guard_t[:4]
    pa.pa_v2_build_tables(i32([0, 0]).cuda(), i32([3, 3]).cuda(), table.cuda(), 2, t, status=st)
    torch.cuda.synchronize()
    assert int(st) & pa.DEVICE_BAD_LENGTH
    assert guard_i[3:].eq(-77).all() and guard_t[4:].eq(-77).all()
    assert t.indptr.tolist() == [0, 2, 4] and t.qo_indptr.tolist() == [0, 3, 4]


def test_tables_empty_free_list_is_one_that_ran_out():
    """No page left: the pages are -1 and reported, and what stood in the table's unused entries (here another
    request's pages) is not taken for them."""
    stale = torch.tensor([[3, 9, 3, 9], [5, 6, 5, 6]], dtype=I32)
    pool = torch.arange(12, dtype=I32, device="cuda")
    for free in (torch.empty(0, dtype=I32, device="cuda"), pool[12:], pool[5:5]):
        st = status_word()
        t = _fresh_tables(2, 8, 8, 0)
        d = stale.cuda()
        pa.pa_v2_build_tables(i32([3, 4]).cuda(), i32([4, 1]).cuda(), d, 2, t, free_pages=free, status=st)
        torch.cuda.synchronize()
        assert int(st) == pa.DEVICE_NO_PAGES
        assert int(t.pages_needed) == 3
        assert d.tolist() == [[3, 9, -1, -1], [5, 6, -1, 6]]
        assert t.indices[:7].tolist() == [3, 9, -1, -1, 5, 6, -1]
        assert t.slots[:5].tolist() == [9 * 2 + 1, -1, -1, -1, -1]
    # one page to take (two cached tokens fill the second request's first page), then none: an empty list is enough
    st = status_word()
    pa.pa_v2_build_tables(i32([3, 2]).cuda(), i32([1, 2]).cuda(), stale.cuda(), 2, t, free_pages=pool[:0], status=st)
    assert int(st) == pa.DEVICE_NO_PAGES and int(t.pages_needed) == 1
    assert t.slots[:3].tolist() == [9 * 2 + 1, -1, -1]
    st = status_word()
    pa.pa_v2_build_tables(i32([3, 3]).cuda(), i32([1, 1]).cuda(), stale.cuda(), 2, t, free_pages=pool[:0], status=st)
    assert int(st) == 0 and int(t.pages_needed) == 0 and t.slots[:2].tolist() == [9 * 2 + 1, 6 * 2 + 1]


def test_tables_bad_parents_become_roots():
    st = status_word()
    t = _fresh_tables(1, 4, 5, 1)
    pa.pa_v2_build_tables(i32([3]).cuda(), i32([5]).cuda(), torch.arange(4, dtype=I32, device="cuda").reshape(1, 4), 4, t,
                          parents=i32([-1, 1, 0, 7, -5]).cuda(), status=st)
    torch.cuda.synchronize()
    assert int(st) & pa.DEVICE_BAD_TREE
    assert t.tree_mask.flatten().tolist() == [1, 2, 5, 8, 16]
    assert t.positions.tolist() == [3, 3, 4, 3, 3]


def test_tables_in_a_replayed_graph_follow_the_lengths():
    case = _tables_case(11, 4, 16, 300, 9, True, 0, True, 6)
    cached, fresh, parents, table, free, cap_i, cap_t, words = case
    fresh = [3, 9, 1, 5]
    parents = [R.random_tree(random.Random(i), n) for i, n in enumerate(fresh)]
    cap_t, cap_i, words = 24, 200, 1
    table = torch.arange(4 * 40, dtype=I32).reshape(4, 40)
    free = torch.arange(1000, 1100, dtype=I32)
    dc, dn, dt, df = i32(cached).cuda(), i32(fresh).cuda(), table.cuda(), free.cuda()
    dp = i32([p for ps in parents for p in ps] + [-1] * (cap_t - sum(fresh))).cuda()
    t = _fresh_tables(4, cap_i, cap_t, words)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        pa.pa_v2_build_tables(dc, dn, dt, 16, t, free_pages=df, parents=dp)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pa.pa_v2_build_tables(dc, dn, dt, 16, t, free_pages=df, parents=dp)
    for step in range(3):
        cached = [c + 40 * step for c in cached]
        dc.copy_(i32(cached))
        dt.copy_(table)
        for f in FIELDS:
            getattr(t, f).fill_(-77)
        g.replay()
        _check_tables(t, dt, R.tables_ref(cached, fresh, table, free, parents, 16, 0, words), cap_t)


# ---------------------------------------------------------------------------
# q/k norm, rotation, append
# ---------------------------------------------------------------------------

def _qk_case(T, hq, hkv, D, rot, dtype, norm, page_size, seed, pos_hi=5000, packed=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, hq + 2 * hkv, D, generator=g) * 1.5).to(dtype).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pages = -(-(T + 7) // page_size) + 1
    slots = torch.randperm(pages * page_size, generator=g)[:T].to(I32)
    pos = torch.randint(0, pos_hi, (T,), generator=g).to(I32)
    half = rot // 2
    freq = torch.tensor([10000.0 ** (-j / max(half, 1)) for j in range(half)], dtype=torch.float32)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)] if norm else [None, None]
    kp = torch.randn(pages, page_size, hkv, D, generator=g).to(dtype)
    vp = torch.randn(pages, page_size, hkv, D, generator=g).to(dtype)
    return q, k, v, pos, slots, freq, w, kp, vp


def _check_qk(case, interleaved, q_dtype, eps=1e-5, status=None, stream=None):
    q, k, v, pos, slots, freq, w, kp, vp = case
    dk, dv = kp.cuda(), vp.cuda()
    out = torch.full(q.shape, 7.0, dtype=q_dtype, device="cuda")
    pa.pa_v2_qk_rope_append(q, k, v, pos.cuda(), slots.cuda(), freq.cuda() if len(freq) else None, dk, dv, q_out=out,
                            q_weight=w[0].cuda() if w[0] is not None else None,
                            k_weight=w[1].cuda() if w[1] is not None else None, eps=eps, interleaved=interleaved,
                            status=status, stream=stream)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < kp.shape[0] * kp.shape[1])
    qr, qm = R.rope_ref(q.cpu(), w[0], eps, pos, freq, interleaved)
    kr, km = R.rope_ref(k.cpu(), w[1], eps, pos, freq, interleaved)
    got = out.cpu().double()
    assert ((got - qr).abs()[live] <= R.rope_tolerance(qr, qm, q_dtype)[live]).all(), (got - qr).abs()[live].max()
    assert got[~live].eq(7.0).all()
    rows = slots[live].long()
    gk, gv = dk.cpu().flatten(0, 1), dv.cpu().flatten(0, 1)
    tol = R.rope_tolerance(kr, km, kp.dtype)[live]
    assert ((gk[rows].double() - kr[live]).abs() <= tol).all()
    assert torch.equal(gv[rows], v.cpu()[live])
    rest = torch.ones(gk.shape[0], dtype=torch.bool)
    rest[rows] = False
    assert torch.equal(gk[rest], kp.flatten(0, 1)[rest]) and torch.equal(gv[rest], vp.flatten(0, 1)[rest])


@pytest.mark.parametrize("dtype,q_dtype", [(torch.float16, torch.float16), (torch.float16, torch.float32),
                                           (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                           (torch.float32, torch.float32)])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 32, False), (64, 64, False),
                                               (64, 32, True), (64, 16, False), (128, 96, False), (64, 0, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_matches_the_definition(dtype, q_dtype, D, rot, interleaved, norm):
    _check_qk(_qk_case(5, 6, 2, D, rot, dtype, norm, 16, D + rot), interleaved, q_dtype)


@pytest.mark.parametrize("T,hq,hkv,page_size,packed", [(1, 1, 1, 1, True), (1, 32, 8, 16, True), (37, 28, 4, 5, False),
                                                       (3, 40, 40, 48, True), (130, 7, 1, 256, True), (2, 64, 1, 8, False)])
def test_qk_head_counts_lengths_and_strides(T, hq, hkv, page_size, packed):
    _check_qk(_qk_case(T, hq, hkv, 128, 128, torch.bfloat16, True, page_size, T + hq, packed=packed), False,
              torch.bfloat16)


def test_qk_far_positions_keep_their_angles():
    case = list(_qk_case(6, 2, 1, 64, 64, torch.float32, False, 4, 3))
    case[3] = i32([0, 1, 999_983, 16_777_217, 1 << 30, 2**31 - 1])
    _check_qk(case, False, torch.float32)


def test_qk_negative_positions_turn_the_other_way():
    case = list(_qk_case(4, 2, 1, 64, 64, torch.float32, False, 4, 3))
    case[3] = i32([-1, -77, 5, -100_000])
    _check_qk(case, True, torch.float32)


def test_qk_only_one_weight():
    case = list(_qk_case(4, 3, 3, 64, 64, torch.float16, True, 4, 9))
    for keep in (0, 1):
        w = [None, None]
        w[keep] = case[6][keep]
        _check_qk((*case[:6], w, *case[7:]), True, torch.float16)


def test_qk_padding_and_bad_slots_are_skipped():
    case = list(_qk_case(9, 4, 2, 128, 128, torch.float16, True, 8, 21))
    slots = case[4]
    slots[2] = -1
    slots[8] = -5
    st = status_word()
    _check_qk(case, False, torch.float16, status=st)
    assert int(st) == 0
    slots[5] = case[7].shape[0] * 8
    _check_qk(case, False, torch.float16, status=st)
    assert int(st) == pa.DEVICE_BAD_SLOT


def test_qk_rows_of_zeros_and_large_values():
    case = list(_qk_case(3, 2, 1, 64, 64, torch.bfloat16, True, 4, 5))
    case[0][0] = 0
    case[0][1] = 3e4
    _check_qk(case, False, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 32), (64, 48), (128, 0)])
def test_qk_infinities_beside_elements_that_are_not_rotated(D, rot, interleaved, dtype):
    q, k, v, pos, slots, freq, w, kp, vp = _qk_case(6, 4, 2, D, rot, dtype, False, 16, 13)
    for x in (q, k):
        x[0, 0, rot], x[1, 1, rot + 3], x[2, 0, D - 1] = math.inf, math.nan, -math.inf
    dk, dv = kp.cuda(), vp.cuda()
    out = pa.pa_v2_qk_rope_append(q, k, v, pos.cuda(), slots.cuda(), freq.cuda() if rot else None, dk, dv,
                                  interleaved=interleaved)
    assert torch.equal(out[..., rot:].nan_to_num(nan=-3.0), q[..., rot:].nan_to_num(nan=-3.0))
    assert out[..., :rot].isfinite().all()
    got = dk.flatten(0, 1)[slots.long().cuda()]
    assert torch.equal(got[..., rot:].nan_to_num(nan=-3.0), k[..., rot:].nan_to_num(nan=-3.0))
    assert got[..., :rot].isfinite().all()


def test_qk_empty_call_and_default_output():
    q, k, v, pos, slots, freq, w, kp, vp = _qk_case(4, 4, 2, 64, 64, torch.float16, False, 4, 1)
    e = torch.zeros(0, dtype=I32, device="cuda")
    out = pa.pa_v2_qk_rope_append(q[:0], k[:0], v[:0], e, e, freq.cuda(), kp.cuda(), vp.cuda())
    assert out.shape == (0, 4, 64) and out.dtype == torch.float16
    out = pa.pa_v2_qk_rope_append(q, k, v, pos.cuda(), slots.cuda(), None, kp.cuda(), vp.cuda(), q_dtype=torch.float32)
    assert torch.equal(out, q.float())


def test_qk_refuses_what_it_cannot_pass_on():
    q, k, v, pos, slots, freq, w, kp, vp = _qk_case(4, 4, 2, 64, 64, torch.float16, True, 4, 1)
    good = dict(q=q, k=k, v=v, positions=pos.cuda(), slots=slots.cuda(), inv_freq=freq.cuda(), k_pool=kp.cuda(),
                v_pool=vp.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda())
    for change, words in ((dict(k=k.flatten(1)), r"k must be \[4, heads, 64\], got \[4, 128\]"),
                          (dict(v=v[:, 0]), r"v must be \[4, heads, 64\], got \[4, 64\]"),
                          (dict(q=q[0]), "q must be"), (dict(q=q[None]), "q must be"), (dict(k=k[None]), "k must be"),
                          (dict(k=k.float()), "k must be torch.float16"), (dict(v=v.cpu()), "v must be a CUDA tensor"),
                          (dict(k=k[:3]), "k must be"), (dict(k=k[..., ::2]), "k must be"),
                          (dict(v=v.transpose(0, 1)), "v must be"), (dict(v=v[:, :1]), "k, v and the pools must agree"),
                          (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), "must be contiguous"),
                          (dict(slots=slots.cuda().long()), "slots must be torch.int32"),
                          (dict(positions=pos.cuda()[:2]), "positions must hold 4 elements"),
                          (dict(inv_freq=freq.cuda().half()), "inv_freq must be torch.float32"),
                          (dict(q_weight=w[0].cuda()[:32]), "q_weight must hold 64 elements"),
                          (dict(q_out=torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")), "q_out must be")):
        with pytest.raises(ValueError, match=words):
            pa.pa_v2_qk_rope_append(**{**good, **change})
    assert pa.pa_v2_qk_rope_append(**good).shape == (4, 4, 64)


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------

def _tree_case(seed, reqs, hq, hkv, D, page_size, dtype, fpos=None, trees=None, chain=False, slack=3, words=None):
    """reqs: [(context, new)]; trees: per-request parent lists (random when None)."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    fpos = fpos or [0] * len(reqs)
    lpl, pages = [], []
    for (c, n), f in zip(reqs, fpos):
        end = c + n + f if c + n else 0
        pages.append(-(-end // page_size))
        lpl.append((end - 1) % page_size + 1 if end else 0)
    P = sum(pages) + slack
    kp = torch.randn(P, page_size, hkv, D, generator=g).to(dtype)
    vp = torch.randn(P, page_size, hkv, D, generator=g).to(dtype)
    idx = torch.randperm(P, generator=g)[:sum(pages)].to(I32)
    indptr = i32([sum(pages[:i]) for i in range(len(pages) + 1)])
    qo = i32([sum(n for _, n in reqs[:i]) for i in range(len(reqs) + 1)])
    T = int(qo[-1])
    q = (1.5 * torch.randn(T, hq, D, generator=g)).to(dtype)
    mask = None
    if not chain:
        trees = trees or [R.random_tree(rng, n) for _, n in reqs]
        words = words or -(-max(max((n for _, n in reqs), default=1), 1) // 32)
        mask = R.tree_mask(trees, words)
    return dict(q=q, kp=kp, vp=vp, idx=idx, indptr=indptr, lpl=i32(lpl),
                fpo=i32(f if c + n else 0 for (c, n), f in zip(reqs, fpos)), qo=qo, mask=mask, scale=D ** -0.5)


def _run_tree(c, pad=0, status=None, **kw):
    T, hq, D = c["q"].shape
    q = torch.cat((c["q"], torch.full((pad, hq, D), float("nan"), dtype=c["q"].dtype))).cuda()
    mask = c["mask"]
    if mask is not None and pad:
        mask = torch.cat((mask, torch.full((pad, mask.shape[1]), -1, dtype=I32)))
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    pa.pa_v2_tree_attention(q, c["kp"].cuda(), c["vp"].cuda(), c["idx"].cuda(), c["indptr"].cuda(), c["lpl"].cuda(),
                            c["fpo"].cuda(), c["qo"].cuda(), c["scale"], tree_mask=mask.cuda() if mask is not None else None,
                            out=out, lse2_out=lse, status=status, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def _check_tree(c, pad=0, **kw):
    st = status_word()
    out, lse = _run_tree(c, pad, st, **kw)
    assert int(st) == 0, int(st)
    T = c["q"].shape[0]
    ro, rl, to, tl = R.attention_ref(c["q"], c["kp"], c["vp"], c["idx"], c["indptr"], c["lpl"], c["fpo"], c["qo"],
                                     c["scale"], c["mask"])
    assert out[T:].eq(5.0).all() and lse[T:].eq(5.0).all()
    out, lse = out[:T].double(), lse[:T].double()
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert out[empty].eq(0).all()
    eo, el = (out - ro).abs(), (lse - rl).abs()[~empty]
    assert (eo <= to).all(), f"out off by {eo.max()} where {to.flatten()[eo.argmax()]} is allowed"
    assert (el <= tl[~empty]).all(), f"lse2 off by {el.max()}"
    return out, lse


DT = [torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("reqs", [[(0, 1)], [(1, 1)], [(0, 7)], [(127, 1)], [(128, 1)], [(129, 4)], [(500, 33), (0, 2), (64, 64)],
                                  [(1000, 64)], [(3, 0), (300, 5), (0, 0), (17, 17)]])
def test_tree_lengths(reqs, D, dtype, chain):
    _check_tree(_tree_case(len(reqs) + D, reqs, 8, 2, D, 16, dtype, chain=chain))


@pytest.mark.parametrize("page_size", [1, 2, 3, 5, 7, 8, 12, 15, 16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("mid", [False, True])
def test_tree_page_sizes_and_mid_page_windows(page_size, mid):
    fpos = [page_size - 1, page_size // 2, 0] if mid else None
    _check_tree(_tree_case(page_size, [(300, 9), (40, 31), (700, 3)], 4, 2, 128, page_size, torch.bfloat16, fpos=fpos))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (8, 8), (12, 4), (16, 1), (40, 8), (64, 1)])
def test_tree_head_groups(hq, hkv):
    _check_tree(_tree_case(hq, [(200, 13), (90, 40)], hq, hkv, 64, 16, torch.float16))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,chain", [(31, False), (32, False), (33, False), (65, False), (129, True), (200, False), (300, True)])
def test_tree_many_new_tokens(n, chain, dtype):
    _check_tree(_tree_case(n, [(150, n), (0, n)], 4, 1, 128, 16, dtype, chain=chain))


@pytest.mark.parametrize("dtype", DT)
def test_tree_long_context_split_over_the_machine(dtype):
    _check_tree(_tree_case(8, [(6000, 6), (2500, 2)], 4, 2, 128, 16, dtype))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("reqs,hq,hkv,D,chain,page_size", [
    ([(4095, 20)] * 3, 32, 8, 128, True, 16),            # runs of several tiles, one tile of query rows
    ([(4000, 64), (1, 3), (2500, 64)], 32, 8, 128, False, 16),   # two tiles of query rows
    ([(3000, 37), (2900, 8)], 32, 8, 128, False, 5),     # the same through the gathering loader
    ([(700, 1)] * 60, 8, 8, 128, True, 16),              # several whole heads per run
    ([(300, 1), (90, 2)] * 90, 4, 2, 64, True, 8),
    ([(20000, 3)], 4, 1, 64, False, 64)])
def test_tree_runs_of_several_tiles_and_pieces(reqs, hq, hkv, D, chain, page_size, dtype):
    _check_tree(_tree_case(D + len(reqs), reqs, hq, hkv, D, page_size, dtype, chain=chain))


@pytest.mark.parametrize("reqs,hq,hkv,chain,page_size", [
    ([(9000, 200)], 8, 2, False, 16),                    # four blocks of query rows, the keys cut into segments
    ([(9000, 200), (50, 1), (3000, 90)], 8, 2, True, 16),
    ([(6000, 330)], 8, 2, True, 3),
    ([(0, 700)], 8, 2, True, 16)])                       # nothing but new tokens: blocks that stop at their last one
def test_tree_several_blocks_of_query_rows(reqs, hq, hkv, chain, page_size):
    _check_tree(_tree_case(len(reqs) + page_size, reqs, hq, hkv, 64, page_size, torch.float16, chain=chain))


def test_tree_many_ragged_requests():
    rng = random.Random(4)
    reqs = [(rng.choice([0, 1, 15, 16, rng.randint(0, 700)]), rng.randint(0, 9)) for _ in range(90)]
    _check_tree(_tree_case(4, reqs, 4, 2, 64, 16, torch.bfloat16))


def test_tree_more_requests_than_threads():
    rng = random.Random(9)
    reqs = [(rng.randint(0, 40), rng.randint(0, 2)) for _ in range(1100)]
    _check_tree(_tree_case(9, reqs, 2, 1, 64, 16, torch.float16))


def test_tree_padded_rows_are_left_alone():
    _check_tree(_tree_case(2, [(100, 5), (60, 9)], 8, 2, 128, 16, torch.float16), pad=13)
    _check_tree(_tree_case(2, [(100, 5), (60, 9)], 8, 2, 128, 16, torch.float16, chain=True), pad=13)


def test_tree_masks_that_leave_rows_empty():
    c = _tree_case(6, [(0, 12), (200, 12), (0, 40)], 8, 2, 128, 16, torch.bfloat16)
    c["mask"][3] = 0
    c["mask"][12 + 5] = 0
    c["mask"][24:64] = 0
    c["mask"][40, 1] = 1 << 4
    out, lse = _check_tree(c)
    assert (lse[3] == -math.inf).all() and (lse[24:40] == -math.inf).all() and (lse[12 + 5] != -math.inf).all()


def test_tree_general_masks_and_all_bits():
    c = _tree_case(61, [(70, 20), (5, 33)], 4, 2, 64, 16, torch.float16)
    g = torch.Generator().manual_seed(0)
    c["mask"] = torch.randint(-2**31, 2**31 - 1, c["mask"].shape, generator=g).to(I32)   # bits past n are ignored
    _check_tree(c)
    c["mask"].fill_(-1)
    _check_tree(c)


def test_tree_mask_without_words_is_refused():
    """An empty mask is not a chain: its rows show nothing to anybody, and nothing can hold that."""
    c = _tree_case(63, [(70, 3)], 4, 2, 64, 16, torch.float16)
    with pytest.raises(ValueError, match="at least one word"):
        _run_tree(dict(c, mask=torch.zeros(3, 0, dtype=I32)))
    with pytest.raises(ValueError, match="at least one word"):
        _run_tree(dict(c, mask=c["mask"].flatten()))
    t = _fresh_tables(1, 4, 4, 1)
    t.tree_mask = t.tree_mask[:, :0]
    with pytest.raises(ValueError, match="at least one word"):
        pa.pa_v2_build_tables(i32([3]).cuda(), i32([2]).cuda(), torch.zeros(1, 4, dtype=I32, device="cuda"), 4, t)


def test_tree_wider_mask_rows_than_needed():
    _check_tree(_tree_case(62, [(70, 20), (5, 33)], 4, 2, 64, 16, torch.float16, words=32))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_tree_nothing_behind_the_mask_reaches_a_result(bad, page_size, dtype):
    c = _tree_case(33, [(100, 20), (300, 9), (0, 3)], 8, 2, 128, page_size, dtype, fpos=[3, 0, 1])
    kp, vp = c["kp"].flatten(0, 1), c["vp"].flatten(0, 1)
    used = torch.zeros(kp.shape[0], dtype=torch.bool)
    drafted = []
    for r in range(3):
        ids = c["idx"][int(c["indptr"][r]):int(c["indptr"][r + 1])].long()
        rows = (ids[:, None] * page_size + torch.arange(page_size)).reshape(-1)
        rows = rows[int(c["fpo"][r]):(len(ids) - 1) * page_size + int(c["lpl"][r])]
        used[rows] = True
        drafted.append(rows[len(rows) - int(c["qo"][r + 1] - c["qo"][r]):])
    kp[~used] = bad                    # stale rows of the pages, and pages of nobody
    vp[~used] = bad
    _check_tree(c)
    # a new token nobody but itself sees: its row may be anything, the others stay what they were
    lone = int(drafted[0][7])
    c["mask"][:20] &= ~(1 << 7)
    c["mask"][7] = 1 << 7
    kp[lone], vp[lone] = bad, bad
    st = status_word()
    out, lse = _run_tree(c, 0, st)
    assert int(st) == 0
    ref = dict(c, kp=c["kp"].clone(), vp=c["vp"].clone())
    ref["kp"].flatten(0, 1)[lone], ref["vp"].flatten(0, 1)[lone] = 0, 0
    ro, rl, to, tl = R.attention_ref(ref["q"], ref["kp"], ref["vp"], c["idx"], c["indptr"], c["lpl"], c["fpo"], c["qo"],
                                     c["scale"], c["mask"])
    keep = torch.arange(len(ro)) != 7
    assert ((out.double() - ro).abs()[keep] <= to[keep]).all()
    assert ((lse.double() - rl).abs()[keep] <= tl[keep]).all()


@pytest.mark.parametrize("dtype", DT)
def test_tree_visible_nan_and_infinite_values_do_reach_their_rows(dtype):
    c = _tree_case(35, [(40, 6)], 4, 1, 128, 16, dtype, trees=[[-1, 0, 0, 1, 1, 2]])
    ids = c["idx"].long()
    rows = (ids[:, None] * 16 + torch.arange(16)).reshape(-1)
    vp = c["vp"].flatten(0, 1)
    vp[int(rows[40 + 1]), 0, 3] = float("inf")       # new token 1: seen by 1, 3, 4
    vp[int(rows[40 + 2]), 0, 5] = float("nan")       # new token 2: seen by 2, 5
    out, lse = _run_tree(c)
    assert torch.isfinite(lse).all()
    for t in range(6):
        assert torch.isinf(out[t, :, 3]).all() == (t in (1, 3, 4))
        assert torch.isnan(out[t, :, 5]).all() == (t in (2, 5))
        others = [d for d in range(128) if d not in (3, 5)]
        assert torch.isfinite(out[t][:, others]).all()


def _check_tree_with_nonfinite_values(c):
    """As _check_tree, where visible values are NaN or infinite: those of the definition have to come out, in the
    elements they belong to, and every other element is compared as ever."""
    st = status_word()
    out, lse = _run_tree(c, 0, st)
    assert int(st) == 0
    finite = dict(c, vp=torch.where(c["vp"].isfinite(), c["vp"], torch.zeros_like(c["vp"])))
    args = (c["idx"], c["indptr"], c["lpl"], c["fpo"], c["qo"], c["scale"], c["mask"])
    ro = R.attention_ref(c["q"], c["kp"], c["vp"], *args)[0]
    rf, rl, to, tl = R.attention_ref(c["q"], c["kp"], finite["vp"], *args)
    out, lse = out.double(), lse.double()
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and out[empty].eq(0).all()
    assert ((lse - rl).abs()[~empty] <= tl[~empty]).all()
    assert torch.equal(out.isnan(), ro.isnan())
    assert torch.equal(out == math.inf, ro == math.inf) and torch.equal(out == -math.inf, ro == -math.inf)
    fin = ro.isfinite()
    assert ((out - rf).abs()[fin] <= to[fin]).all()
    return ro


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("copies", [1, 16])
@pytest.mark.parametrize("hq,n", [(8, 12), (2, 100), (8, 48)])   # up to 48, 100 and 192 rows a block: joined streams, two tiles
def test_tree_rows_that_see_nothing_beside_rows_that_see_infinities(hq, n, copies, page_size, dtype):
    """No context: a token without a mask bit sees nothing at all, in the same warp as tokens that see a NaN or an
    infinity; a drafted tree padded with empty rows looks like this."""
    c = _tree_case(81, [(0, n)] * copies, hq, 2, 64, page_size, dtype, fpos=[min(4, page_size - 1)] * copies)
    vp = c["vp"].flatten(0, 1)
    for r in range(copies):
        ids = c["idx"][int(c["indptr"][r]):int(c["indptr"][r + 1])].long()
        rows = (ids[:, None] * page_size + torch.arange(page_size)).reshape(-1)[int(c["fpo"][r]):]
        vp[int(rows[2]), 0, 5] = math.inf
        vp[int(rows[3]), 1, 63] = math.nan
        vp[int(rows[n - 1]), 0, 33] = -math.inf
        c["mask"][r * n + 1:r * n + n:3] = 0
    ref = _check_tree_with_nonfinite_values(c)
    assert (ref == math.inf).any() and (ref == -math.inf).any() and ref.isnan().any()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("copies", [1, 12])
def test_tree_infinities_of_rows_whose_keys_all_lie_in_one_tile(copies, page_size, dtype):
    """128 rows a block, two or three key tiles in one piece (two streams, joined): tokens that see only themselves, in
    the first tile or in the second, and an infinity or a NaN there.  12 requests: 192 or 288 units, so that a CTA
    takes a whole block."""
    first, n = page_size - 1, 128 - (page_size - 1) % 4
    c = _tree_case(83, [(0, n)] * copies, 8, 8, 64, page_size, dtype, fpos=[first] * copies)
    vp = c["vp"].flatten(0, 1)
    for r in range(copies):
        ids = c["idx"][int(c["indptr"][r]):int(c["indptr"][r + 1])].long()
        rows = (ids[:, None] * page_size + torch.arange(page_size)).reshape(-1)[int(c["fpo"][r]):]
        for token, element, value in ((5, 1, math.inf), (n - 1, 2, math.inf), (n - 2, 62, -math.inf), (9, 3, math.nan)):
            c["mask"][r * n:(r + 1) * n, token // 32] &= ~(1 << token % 32) if token % 32 < 31 else 2**31 - 1
            c["mask"][r * n + token] = i32(R.words_of(1 << token, 4))
            vp[int(rows[token]), 1, element] = value
    ref = _check_tree_with_nonfinite_values(c)
    assert ref.isinf().any() and ref.isnan().any()


def test_tree_chain_cut_behind_its_first_tile_beside_infinities():
    """One block of 200 tokens of a chain without context: the last tile may stand as a piece of its own, in which the
    tokens before it see nothing and those behind it, in the same warp, an infinity."""
    c = _tree_case(82, [(0, 200)], 1, 1, 128, 16, torch.bfloat16, chain=True)
    rows = (c["idx"].long()[:, None] * 16 + torch.arange(16)).reshape(-1)
    vp = c["vp"].flatten(0, 1)
    vp[int(rows[130]), 0, 7], vp[int(rows[199]), 0, 8], vp[int(rows[3]), 0, 9] = math.inf, math.nan, -math.inf
    _check_tree_with_nonfinite_values(c)


@pytest.mark.parametrize("dtype", DT)
def test_tree_sharp_and_flat_scores(dtype):
    c = _tree_case(36, [(900, 8)], 4, 2, 128, 16, dtype)
    # keys that climb along the context: the running maximum rises tile after tile
    kp = c["kp"].flatten(0, 1)
    rows = (c["idx"].long()[:, None] * 16 + torch.arange(16)).reshape(-1)[:908]
    ramp = torch.linspace(0, 6, 908)
    kp[rows] = (kp[rows].float() + ramp[:, None, None] * c["q"][0].float().reshape(2, 2, 128).mean(1)).to(dtype)
    _check_tree(c)
    kp[rows] = kp[rows].flip(0)
    _check_tree(c)
    c["q"] = torch.zeros_like(c["q"])                # all scores equal: the mean of v
    _check_tree(c)


def test_tree_scores_far_below_the_maximum_still_count():
    # one key far above the rest: the others' weights are below the 16-bit type's normal range
    c = _tree_case(37, [(4000, 2)], 2, 1, 64, 16, torch.float16)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][:, :, 0] = 8.0
    rows = (c["idx"].long()[:, None] * 16 + torch.arange(16)).reshape(-1)
    kp, vp = c["kp"].flatten(0, 1), c["vp"].flatten(0, 1)
    kp[rows[5], 0, 0] += 12.0
    vp[:] = 1.0
    vp[rows[5]] = -1.0
    _check_tree(c)


def test_tree_negative_and_zero_scale():
    c = _tree_case(38, [(100, 9)], 4, 2, 64, 16, torch.float16)
    for scale in (0.0, -0.2):
        c["scale"] = scale
        st = status_word()
        out, lse = _run_tree(c, 0, st)
        ro, rl, to, tl = R.attention_ref(c["q"], c["kp"], c["vp"], c["idx"], c["indptr"], c["lpl"], c["fpo"], c["qo"],
                                         scale, c["mask"])
        tol = R.attention_ref(c["q"], c["kp"], c["vp"], c["idx"], c["indptr"], c["lpl"], c["fpo"], c["qo"], 0.2,
                              c["mask"])
        assert ((out.double() - ro).abs() <= to.abs() + tol[2]).all()
        assert ((lse.double() - rl).abs() <= tol[3]).all()


@pytest.mark.parametrize("scale,size", [(1e-31, 2.0 ** 50), (1e-36, 2.0 ** 58)])
def test_tree_tiny_scales_of_large_scores(scale, size):
    """Scores of about one out of products of 1e31 and 1e36, which f32 and bf16 hold."""
    c = _tree_case(39, [(300, 9)], 4, 2, 64, 16, torch.bfloat16)
    c["scale"] = float(torch.tensor(scale, dtype=torch.float32))
    c["q"] = (c["q"].float() * size).to(torch.bfloat16)
    c["kp"] = (c["kp"].float() * (0.3 / scale / size)).to(torch.bfloat16)
    _, lse = _check_tree(c)
    assert lse.std() > 0.5


def test_tree_bad_tables_are_contained_and_reported():
    base = _tree_case(40, [(100, 6), (50, 4), (30, 5)], 4, 2, 64, 16, torch.float16)
    ref = _check_tree(base)

    def run(**change):
        c = dict(base, **change)
        st = status_word()
        out, lse = _run_tree(c, 0, st)
        return out.double(), lse.double(), int(st)

    def others_ok(out, lse, bad):
        keep = [t for t in range(15) if t not in bad]
        assert (out[keep] - ref[0][keep]).abs().max() <= 2e-3 and (lse[keep] - ref[1][keep]).abs().max() <= 1e-3

    idx = base["idx"].clone()
    idx[int(base["indptr"][1])] = base["kp"].shape[0] + 3          # request 1's first page id out of range
    out, lse, st = run(idx=idx)
    assert st == pa.DEVICE_BAD_PAGE
    others_ok(out, lse, range(6, 10))
    assert torch.isfinite(out).all()
    idx[int(base["indptr"][1])] = -1
    out, lse, st = run(idx=idx)
    assert st == pa.DEVICE_BAD_PAGE
    others_ok(out, lse, range(6, 10))
    lpl = base["lpl"].clone()
    lpl[0] = 17
    out, lse, st = run(lpl=lpl)
    assert st == pa.DEVICE_BAD_TREE
    others_ok(out, lse, range(0, 6))
    assert out[:6].eq(0).all() and (lse[:6] == -math.inf).all()
    fpo = base["fpo"].clone()
    fpo[2] = -1
    out, lse, st = run(fpo=fpo)
    assert st == pa.DEVICE_BAD_TREE
    others_ok(out, lse, range(10, 15))
    indptr = base["indptr"].clone()
    indptr[3] = base["idx"].numel() + 100
    out, lse, st = run(indptr=indptr)
    assert st == pa.DEVICE_BAD_SLOT
    others_ok(out, lse, range(10, 15))
    assert out[10:].eq(0).all() and (lse[10:] == -math.inf).all()
    qo = base["qo"].clone()
    qo[3] = 99
    out, lse, st = run(qo=qo)
    assert st == pa.DEVICE_BAD_INDPTR
    others_ok(out, lse, range(10, 15))
    assert out[10:].eq(5.0).all()


def test_tree_tables_that_claim_pages_and_tokens_again_stay_in_bounds():
    """Prefix sums that fall and rise again: the falling requests are refused, the others stand on their own."""
    base = _tree_case(47, [(900, 6), (50, 4), (700, 5)], 4, 2, 64, 16, torch.float16)
    ref = _check_tree(base)
    one = [int(x) for x in base["indptr"]]
    c = dict(base, indptr=i32([0, one[1], 0, one[1], 0, one[1]]), lpl=i32([int(base["lpl"][0])] * 5),
             fpo=i32([0] * 5), qo=i32([0, 6, 0, 6, 0, 6]))
    st = status_word()
    out, lse = _run_tree(c, 0, st)
    assert int(st) == pa.DEVICE_BAD_INDPTR
    assert (out[:6].double() - ref[0][:6]).abs().max() <= 2e-3 and (lse[:6].double() - ref[1][:6]).abs().max() <= 1e-3
    assert out[6:].eq(5.0).all()


def test_tree_tokens_of_no_request_are_left_alone():
    c = _tree_case(48, [(100, 6), (50, 4)], 4, 2, 64, 16, torch.float16)
    shifted = dict(c, q=torch.cat((c["q"][:3], c["q"])), mask=torch.cat((c["mask"][:3], c["mask"])), qo=c["qo"] + 3)
    ref, got = _run_tree(c), _run_tree(shifted)
    assert got[0][:3].eq(5.0).all() and got[1][:3].eq(5.0).all()
    assert torch.equal(got[0][3:], ref[0]) and torch.equal(got[1][3:], ref[1])


def test_tree_many_requests_with_several_blocks():
    reqs = [(1500, 150), (0, 90), (400, 1)] * 13                # more than a warp's lanes, two blocks each
    _check_tree(_tree_case(49, reqs, 4, 1, 64, 16, torch.bfloat16))
    _check_tree(_tree_case(49, reqs, 4, 1, 64, 16, torch.bfloat16, chain=True))


def test_tree_two_graphs_with_their_own_workspaces_side_by_side():
    cases = [_tree_case(s, [(2000, 30), (300, 64)], 8, 2, 128, 16, torch.float16) for s in (51, 52)]
    refs = [_run_tree(c) for c in cases]
    graphs, outs, keep = [], [], []
    for c in cases:
        d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
        ws = pa.tree_attention_workspace(c["q"].shape[0], 2, 8, 2, 128)
        out, lse = torch.zeros_like(d["q"]), torch.zeros(d["q"].shape[:2], device="cuda")
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            pa.pa_v2_tree_attention(d["q"], d["kp"], d["vp"], d["idx"], d["indptr"], d["lpl"], d["fpo"], d["qo"],
                                    d["scale"], tree_mask=d["mask"], out=out, lse2_out=lse, workspace=ws)
        graphs.append((g, s))
        outs.append((out, lse))
        keep.append((d, ws))
    for _ in range(3):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (out, lse), ref in zip(outs, refs):
            assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])
            out.zero_()


def test_tree_more_new_tokens_than_visible_ones_or_than_mask_bits():
    c = _tree_case(41, [(0, 4), (60, 40)], 4, 2, 64, 16, torch.float16)
    c["lpl"] = i32([2, int(c["lpl"][1])])             # request 0 lists two tokens, has four new ones
    c["mask"] = c["mask"][:, :1].contiguous()         # request 1 has more new tokens than bits
    st = status_word()
    out, lse = _run_tree(c, 0, st)
    assert int(st) == pa.DEVICE_BAD_TREE
    assert out.eq(0).all() and (lse == -math.inf).all()


def test_tree_repeats_itself_exactly():
    c = _tree_case(43, [(3000, 17), (10, 5), (800, 64)], 8, 2, 128, 16, torch.bfloat16)
    a = _run_tree(c)
    for _ in range(3):
        b = _run_tree(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_on_another_stream_with_its_own_buffers():
    c = _tree_case(44, [(700, 9), (65, 3)], 8, 2, 128, 16, torch.float16)
    ref = _run_tree(c)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out, lse = pa.pa_v2_tree_attention(d["q"], d["kp"], d["vp"], d["idx"], d["indptr"], d["lpl"], d["fpo"], d["qo"],
                                           d["scale"], tree_mask=d["mask"], stream=stream)
        s.synchronize()
        assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])


def test_tree_workspace_with_any_contents_and_too_small():
    c = _tree_case(45, [(2000, 9), (65, 3)], 8, 2, 128, 16, torch.float16)
    ref = _run_tree(c)
    ws = pa.tree_attention_workspace(c["q"].shape[0], 2, 8, 2, 128)
    for fill in (0, 255):
        got = _run_tree(c, workspace=ws.fill_(fill))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    with pytest.raises(pa.PaError) as e:
        _run_tree(c, workspace=ws[:ws.numel() - 16])
    assert e.value.status == pa.PA_ECAPACITY


def test_tree_single_tokens_agree_with_the_decode():
    reqs = [(777, 1), (0, 1), (4095, 1)]
    c = _tree_case(46, reqs, 32, 8, 128, 16, torch.float16, chain=True)
    out, lse = _check_tree(c)
    plan = pa.pa_v2_plan(c["indptr"], c["lpl"], c["fpo"], 16, 32, 8, 128, pa.PA_F16,
                         pa.pa_v2_default_target_ctas(32, 8, 128, 16, pa.PA_F16))
    o, l = pa.decode(plan, c["q"].float().cuda(), c["kp"].cuda(), c["vp"].cuda(), c["idx"].cuda(), c["indptr"].cuda(),
                     c["lpl"].cuda(), c["fpo"].cuda(), c["scale"])
    assert (o.cpu().double() - out).abs().max() <= 2e-3 and (l.cpu().double() - lse).abs().max() <= 1e-3


# ---------------------------------------------------------------------------
# sliding windows: every token sees its own
# ---------------------------------------------------------------------------

def _sliding_case(seed, reqs, window, tree, hq, hkv, D, page_size, dtype, words=None):
    """reqs [(cached, new)] whose K and V, new tokens' included, lie in the pools at block_table's pages; seen: the pool
    rows each new token sees."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    cached, fresh = [c for c, _ in reqs], [n for _, n in reqs]
    parents = [R.random_tree(rng, n) for n in fresh] if tree == "random" else \
              [[i - 1 if i % 9 else max(i - 4, -1) for i in range(n)] for n in fresh] if tree == "deep" else None
    width = max(-(-(c + n) // page_size) for c, n in reqs) + 1
    P = len(reqs) * width + 2
    table = torch.randperm(P, generator=g)[:len(reqs) * width].reshape(-1, width).to(I32)
    kp, vp = (torch.randn(P, page_size, hkv, D, generator=g).to(dtype) for _ in range(2))
    q = (1.5 * torch.randn(sum(fresh), hq, D, generator=g)).to(dtype)
    seen = []
    for r, (c, n) in enumerate(reqs):
        row = lambda at: int(table[r, at // page_size]) * page_size + at % page_size
        for i in range(n):
            line = R.ancestors(parents[r] if parents is not None else None, i)
            low = c + len(line) - 1 - window + 1          # its position is c + its depth
            seen.append([row(x) for x in range(max(low, 0), c)] +
                        [row(c + j) for d, j in reversed(list(enumerate(line))) if d < window])
    words = words or (-(-max(fresh) // 32) if tree else 0)
    return dict(cached=cached, fresh=fresh, parents=parents, table=table, kp=kp, vp=vp, q=q, seen=seen, words=words,
                window=window, page_size=page_size, scale=D ** -0.5)


def _sliding_run(c, st, table=None, tables_window=None, kp=None, vp=None):
    """Tables, then attention: (tables, out, lse2)."""
    cap_t = sum(c["fresh"]) + 3
    t = _fresh_tables(len(c["cached"]), c["table"].numel(), cap_t, c["words"])
    packed = i32([p for ps in c["parents"] for p in ps] + [-1] * 3).cuda() if c["parents"] is not None else None
    pa.pa_v2_build_tables(i32(c["cached"]).cuda(), i32(c["fresh"]).cuda(), (c["table"] if table is None else table).cuda(),
                          c["page_size"], t, parents=packed, status=st,
                          **(tables_window if tables_window is not None else dict(sliding_window=c["window"])))
    q = torch.cat((c["q"], torch.full((3, *c["q"].shape[1:]), float("nan"), dtype=c["q"].dtype))).cuda()
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 5.0, device="cuda")
    pa.pa_v2_tree_attention(q, (c["kp"] if kp is None else kp).cuda(), (c["vp"] if vp is None else vp).cuda(), t.indices,
                            t.indptr, t.last_page_len, t.first_page_offset, t.qo_indptr, c["scale"],
                            tree_mask=t.tree_mask, out=out, lse2_out=lse, status=st, sliding_window=c["window"],
                            positions=t.positions)
    torch.cuda.synchronize()
    assert out[-3:].eq(5.0).all() and lse[-3:].eq(5.0).all()
    return t, out[:-3].cpu().double(), lse[:-3].cpu().double()


def _check_sliding(c, ref, got):
    assert ((got[1] - ref[1]).abs() <= ref[3]).all(), (got[1] - ref[1]).abs().max()
    assert ((got[0] - ref[0]).abs() <= ref[2]).all(), (got[0] - ref[0]).abs().max()


SLIDING = [
    ([(5000, 5), (100, 5), (4094, 3)], 4096, None, 8, 2, 128, 16),     # a verified chain
    ([(700, 5), (0, 5), (127, 4), (128, 1), (40, 0)], 128, None, 8, 2, 128, 16),
    ([(700, 64), (126, 64), (3, 64)], 128, "random", 8, 2, 128, 16),
    ([(700, 64), (30, 50)], 20, "deep", 8, 2, 64, 16),                 # trees deeper than the window
    ([(300, 9), (50, 33)], 1, "deep", 4, 2, 64, 5),                    # every token sees itself alone
    ([(300, 9), (0, 30)], 1, None, 4, 2, 64, 16),
    ([(257, 7), (511, 40)], 33, "random", 4, 4, 128, 5),
    ([(900, 300), (0, 290)], 64, None, 4, 1, 64, 16),                  # several blocks, more new tokens than the window
    ([(900, 300), (20, 130)], 500, None, 8, 2, 128, 48),
    ([(2000, 200)], 300, "deep", 4, 1, 64, 256),
    ([(200, 3)] * 70, 100, None, 2, 1, 64, 16),                        # more requests than a warp's lanes
    ([(400, 6)], 100000, "random", 4, 2, 64, 16),                      # a window that never binds
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("reqs,window,tree,hq,hkv,D,page_size", SLIDING)
def test_sliding_step_equals_each_token_alone(reqs, window, tree, hq, hkv, D, page_size, dtype):
    c = _sliding_case(len(reqs) + window, reqs, window, tree, hq, hkv, D, page_size, dtype)
    st = status_word()
    t, out, lse = _sliding_run(c, st)
    assert int(st) == 0
    ref = R.sliding_tables_ref(c["cached"], c["fresh"], c["table"], None, c["parents"], page_size, window, c["words"])
    _check_tables(t, c["table"], ref, sum(c["fresh"]) + 3)
    _check_sliding(c, R.rows_attention_ref(c["q"], c["kp"], c["vp"], c["seen"], c["scale"]), (out, lse))


@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tree", [None, "deep"])
def test_sliding_window_hides_what_lies_before_it(tree, bad, page_size):
    """Keys and values before the window of every token, pages that are gone, and rows that only the first tokens of a
    request still see: none of it reaches a token that does not see it."""
    c = _sliding_case(7, [(700, 40), (300, 7), (60, 12)], 150, tree, 8, 2, 64, page_size, torch.bfloat16)
    ref = R.rows_attention_ref(c["q"], c["kp"], c["vp"], c["seen"], c["scale"])
    used = torch.zeros(c["kp"].shape[0] * page_size, dtype=torch.bool)
    for rows in c["seen"]:
        used[rows] = True
    kp, vp = c["kp"].clone(), c["vp"].clone()
    kp.flatten(0, 1)[~used], vp.flatten(0, 1)[~used] = bad, bad
    st = status_word()
    _check_sliding(c, ref, _sliding_run(c, st, kp=kp, vp=vp)[1:])
    # tables that list every page, those before the window given back already
    gone = c["table"].clone()
    for r, n in enumerate(c["cached"]):
        gone[r, :max(0, n - 149) // page_size] = -1 if r else 10**6
    _check_sliding(c, ref, _sliding_run(c, st, table=gone, tables_window={}, kp=kp, vp=vp)[1:])
    # tables of a window that is wide enough for the longest request
    _check_sliding(c, ref, _sliding_run(c, st, table=gone, tables_window=dict(window=189))[1:])
    assert int(st) == 0
    # what the first token of each request sees last of all: bad for it and for nobody else
    hidden, t0 = set(), 0
    for n in c["fresh"]:
        row = c["seen"][t0][0]
        kp.flatten(0, 1)[row], vp.flatten(0, 1)[row] = bad, bad
        hidden |= {t for t, rows in enumerate(c["seen"]) if row in rows}
        t0 += n
    keep = [t for t in range(len(c["seen"])) if t not in hidden]
    assert len(keep) > 40
    _, out, lse = _sliding_run(c, st, kp=kp, vp=vp)
    assert int(st) == 0
    assert ((out - ref[0]).abs()[keep] <= ref[2][keep]).all() and ((lse - ref[1]).abs()[keep] <= ref[3][keep]).all()
    # a value alone (its key is finite): the tokens that see it get it, in its element
    kp = c["kp"]
    vp = c["vp"].clone()
    vp.flatten(0, 1)[c["seen"][0][0], 1, 9] = bad
    sees = [c["seen"][0][0] in rows for rows in c["seen"]]
    _, out, lse = _sliding_run(c, st, vp=vp)
    assert (~out[:, 4:, 9].isfinite()).all(1).tolist() == sees and (~out[:, 4:, 9].isfinite()).any(1).tolist() == sees
    out[:, 4:, 9] = ref[0][:, 4:, 9]
    _check_sliding(c, ref, (out, lse))


def test_sliding_step_refuses_tables_that_lack_what_its_tokens_see():
    """Tables of the request's last 100 tokens hold 95 earlier ones beside 5 new; the first new one sees 99."""
    c = _sliding_case(9, [(300, 5), (60, 5), (300, 1)], 100, None, 4, 2, 64, 16, torch.float16)
    ref = R.rows_attention_ref(c["q"], c["kp"], c["vp"], c["seen"], c["scale"])
    st = status_word()
    _, out, lse = _sliding_run(c, st, tables_window=dict(window=100))
    assert int(st) == pa.DEVICE_BAD_TREE
    assert out[:5].eq(0).all() and (lse[:5] == -math.inf).all()
    assert ((out - ref[0]).abs()[5:] <= ref[2][5:]).all()            # everything of 60, and a single token's window
    with pytest.raises(ValueError, match="positions"):
        pa.pa_v2_tree_attention(*([torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")] +
                                  [torch.zeros(1, 1, 2, 64, dtype=torch.float16, device="cuda")] * 2 +
                                  [torch.zeros(2, dtype=I32, device="cuda")] * 2 +
                                  [torch.zeros(1, dtype=I32, device="cuda")] * 2 +
                                  [torch.zeros(2, dtype=I32, device="cuda")]), 0.1, sliding_window=3)


def test_sliding_chain_at_once_equals_one_token_at_a_time():
    """The chain of a step against the same tokens appended one by one, each through tables and attention of its own."""
    c = _sliding_case(10, [(500, 6), (130, 6)], 128, None, 8, 2, 128, 16, torch.bfloat16)
    st = status_word()
    _, out, lse = _sliding_run(c, st)
    ref = R.rows_attention_ref(c["q"], c["kp"], c["vp"], c["seen"], c["scale"])
    for i in range(6):
        one = dict(c, cached=[n + i for n in c["cached"]], fresh=[1, 1], q=c["q"][[i, 6 + i]])
        for tables_window in (dict(window=128), dict(sliding_window=128)):
            _, o, l = _sliding_run(one, st, tables_window=tables_window)
            assert ((o - out[[i, 6 + i]]).abs() <= 2 * ref[2][[i, 6 + i]]).all()      # each within its tolerance
            assert ((l - lse[[i, 6 + i]]).abs() <= 2 * ref[3][[i, 6 + i]]).all()
    assert int(st) == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def _dense_step(reqs, trees, x, hist, weights, freq, eps, hq, hkv, D, scale, window):
    """The step from dense histories: per request (k [c, hkv, D], v) in the pool's dtype; x packed projections."""
    G = hq // hkv
    outs, tols = [], []
    t0 = 0
    for (c, n), tree, (kh, vh) in zip(reqs, trees, hist):
        xs = x[t0:t0 + n]
        pos = torch.tensor([c + len(R.ancestors(tree, i)) - 1 for i in range(n)])
        q, _ = R.rope_ref(xs[:, :hq], weights[0], eps, pos, freq, False)
        k, _ = R.rope_ref(xs[:, hq:hq + hkv], weights[1], eps, pos, freq, False)
        q, k = q.to(x.dtype), k.to(x.dtype)
        keys, vals = torch.cat((kh, k)), torch.cat((vh, xs[:, hq + hkv:]))
        lo = max(0, c + n - window) if window else 0
        for i in range(n):
            sees = [j for j in range(lo, c)] + [c + j for j in R.ancestors(tree, i) if c + j >= lo]
            kk, vv = keys[sees].double(), vals[sees].double()
            s = torch.einsum("hgd,khd->hgk", q[i].double().reshape(hkv, G, D), kk) * scale
            p = torch.softmax(s, -1)
            outs.append(torch.einsum("hgk,khd->hgd", p, vv).reshape(hq, D))
            tols.append(torch.einsum("hgk,khd->hgd", p, vv.abs()).reshape(hq, D))
        t0 += n
    return torch.stack(outs), torch.stack(tols)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("window", [0, 150])
def test_a_whole_step_from_lengths_to_outputs(graph, window):
    """Tables, then q/k preparation into the pools, then tree attention: two steps of growing requests, eagerly and
    from one captured graph, against dense attention over each request's own history."""
    dtype, hq, hkv, D, ps, B = torch.bfloat16, 8, 2, 64, 16, 3
    rng = random.Random(77)
    g = torch.Generator().manual_seed(77)
    cap_t, width, P = 40, 40, 200
    freq = torch.tensor([10000.0 ** (-j / 32) for j in range(32)], dtype=torch.float32)
    weights = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)]
    cached = [200, 0, 37]
    table = torch.full((B, width), -1, dtype=I32)
    perm = torch.randperm(P, generator=g).to(I32)
    used = 0
    kp, vp = torch.full((P, ps, hkv, D), float("nan"), dtype=dtype), torch.full((P, ps, hkv, D), float("nan"), dtype=dtype)
    hist = []
    for r, c in enumerate(cached):
        k, v = torch.randn(c, hkv, D, generator=g).to(dtype), torch.randn(c, hkv, D, generator=g).to(dtype)
        for j in range(-(-c // ps)):
            table[r, j] = perm[used]
            used += 1
        for i in range(c):
            kp[table[r, i // ps].long(), i % ps], vp[table[r, i // ps].long(), i % ps] = k[i], v[i]
        hist.append([k, v])
    dk, dv, dtab = kp.cuda(), vp.cuda(), table.cuda()
    dfree = torch.full((P,), -1, dtype=I32, device="cuda")
    dc, dn = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    dpar = torch.full((cap_t,), -1, dtype=I32, device="cuda")
    dx = torch.zeros(cap_t, hq + 2 * hkv, D, dtype=dtype, device="cuda")
    t = pa.StepTables.empty(B, B * width, cap_t, 1)
    st = status_word()
    dq = torch.empty(cap_t, hq, D, dtype=dtype, device="cuda")
    out, lse = torch.empty_like(dq), torch.empty(cap_t, hq, device="cuda")
    ws = pa.tree_attention_workspace(cap_t, B, hq, hkv, D)
    dfreq, dw = freq.cuda(), [w.cuda() for w in weights]

    def step():
        pa.pa_v2_build_tables(dc, dn, dtab, ps, t, free_pages=dfree, parents=dpar, window=window, status=st)
        pa.pa_v2_qk_rope_append(dx[:, :hq], dx[:, hq:hq + hkv], dx[:, hq + hkv:], t.positions, t.slots, dfreq, dk, dv,
                                q_out=dq, q_weight=dw[0], k_weight=dw[1], eps=1e-6, status=st)
        pa.pa_v2_tree_attention(dq, dk, dv, t.indices, t.indptr, t.last_page_len, t.first_page_offset, t.qo_indptr,
                                D ** -0.5, tree_mask=t.tree_mask, out=out, lse2_out=lse, workspace=ws, status=st)

    replay = step
    if graph:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()                                    # empty lengths: nothing is written
        s.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=s):
            step()
        replay = cg.replay
    for _ in range(2):
        fresh = [rng.randint(1, 13) for _ in range(B)]
        trees = [R.random_tree(rng, n) for n in fresh]
        n = sum(fresh)
        x = torch.randn(n, hq + 2 * hkv, D, generator=g).to(dtype)
        dc.copy_(i32(cached))
        dn.copy_(i32(fresh))
        dpar[:n] = i32(p for ps_ in trees for p in ps_).cuda()
        dx[:n] = x.cuda()
        dfree[:P - used] = perm[used:].cuda()
        replay()
        torch.cuda.synchronize()
        assert int(st) == 0
        ref, mean_abs = _dense_step(list(zip(cached, fresh)), trees, x, hist, weights, freq, 1e-6, hq, hkv, D, D ** -0.5,
                                    window)
        # q and k are each rounded once on both sides, possibly to neighbouring values where f32 and f64 straddle a
        # rounding border: a step of eps in q or k moves a score by at most eps * |q||k| * scale (about 2^-7 * 8)
        e = torch.finfo(dtype).eps
        tol = ref.abs() * e / 2 + mean_abs * (e / 2 + 2 * e)
        assert ((out[:n].cpu().double() - ref).abs() <= tol).all()
        # accept one path of each tree (its tokens are the next step's history) and keep the rest out of the cache
        used += int(t.pages_needed)
        t0 = 0
        slots = t.slots.cpu()
        for r in range(B):
            path = sorted(R.ancestors(trees[r], fresh[r] - 1))
            src = slots[t0 + torch.tensor(path)].long()
            dst = slots[t0:t0 + len(path)].long()
            fk, fv = dk.flatten(0, 1), dv.flatten(0, 1)
            fk[dst.cuda()], fv[dst.cuda()] = fk[src.cuda()].clone(), fv[src.cuda()].clone()
            hist[r][0] = torch.cat((hist[r][0], fk[dst.cuda()].cpu()))
            hist[r][1] = torch.cat((hist[r][1], fv[dst.cuda()].cpu()))
            cached[r] += len(path)
            t0 += fresh[r]


def test_tables_feed_the_single_token_decode():
    """One new token per request: the device-made tables and an f32 q drive pa_v2_decode_partial + merge."""
    dtype, hq, hkv, D, ps = torch.float16, 8, 2, 128, 16
    cached = [100, 0, 515]
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(150, generator=g)[:3 * 40].reshape(3, 40).to(I32)
    t = pa.StepTables.empty(3, 120, 3)
    pa.pa_v2_build_tables(i32(cached).cuda(), i32([1, 1, 1]).cuda(), table.cuda(), ps, t)
    kp, vp = torch.randn(150, ps, hkv, D, generator=g).to(dtype).cuda(), torch.randn(150, ps, hkv, D, generator=g).to(dtype).cuda()
    x = torch.randn(3, hq + 2 * hkv, D, generator=g).to(dtype).cuda()
    freq = torch.tensor([10000.0 ** (-j / 64) for j in range(64)], dtype=torch.float32).cuda()
    q = pa.pa_v2_qk_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], t.positions, t.slots, freq, kp, vp,
                                q_dtype=torch.float32)
    ip, lp, fp = t.indptr.cpu(), t.last_page_len.cpu(), t.first_page_offset.cpu()
    assert ip.tolist() == [0, 7, 8, 41] and lp.tolist() == [5, 1, 4]
    plan = pa.pa_v2_plan(ip, lp, fp, ps, hq, hkv, D, pa.PA_F16,
                         pa.pa_v2_default_target_ctas(hq, hkv, D, ps, pa.PA_F16), seq_lens=[101, 1, 516])
    o, l = pa.decode(plan, q, kp, vp, t.indices[:int(ip[-1])], t.indptr, t.last_page_len, t.first_page_offset, D ** -0.5)
    q16 = pa.pa_v2_qk_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], t.positions, t.slots, freq, kp, vp)
    o2, l2 = pa.pa_v2_tree_attention(q16, kp, vp, t.indices, t.indptr, t.last_page_len, t.first_page_offset,
                                     t.qo_indptr, D ** -0.5)
    ro, rl, to, tl = R.attention_ref(q16.cpu(), kp.cpu(), vp.cpu(), t.indices.cpu(), ip, lp, fp, t.qo_indptr.cpu(),
                                     D ** -0.5)
    assert ((o2.cpu().double() - ro).abs() <= to).all() and ((l2.cpu().double() - rl).abs() <= tl).all()
    # the decode reads the unrounded q: one rounding of q apart (2^-11 of scores of size |q||k|/sqrt(D) ~ 12)
    assert (o.cpu().double() - ro).abs().max() <= 2e-2 and (l.cpu().double() - rl).abs().max() <= 2e-2


@pytest.mark.parametrize("page_size", [16, 5])
def test_pools_of_more_elements_than_32_bits_count(page_size):
    hkv, D = 8, 128
    pages = ((1 << 32) // (hkv * D) + (1 << 17)) // page_size
    big_k, big_v = (torch.empty(pages, page_size, hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
    assert big_k.numel() > 1 << 32

    # the small case's pages at the end of the large pools: the same results, bit for bit
    c = _tree_case(71, [(900, 33), (40, 5)], 32, hkv, D, page_size, torch.float16)
    want = _run_tree(c)
    shift = pages - c["kp"].shape[0]
    big_k[shift:], big_v[shift:] = c["kp"].cuda(), c["vp"].cuda()
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    out, lse = pa.pa_v2_tree_attention(d["q"], big_k, big_v, d["idx"] + shift, d["indptr"], d["lpl"], d["fpo"], d["qo"],
                                       d["scale"], tree_mask=d["mask"])
    assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])

    q, k, v, pos, slots, freq, w, kp, vp = _qk_case(70, 32, hkv, D, 128, torch.float16, True, page_size, 72)
    weights = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda())
    dk, dv = kp.cuda(), vp.cuda()
    small = pa.pa_v2_qk_rope_append(q, k, v, pos.cuda(), slots.cuda(), freq.cuda(), dk, dv, **weights)
    shift = pages - kp.shape[0]
    big_k[shift:], big_v[shift:] = kp.cuda(), vp.cuda()
    large = pa.pa_v2_qk_rope_append(q, k, v, pos.cuda(), slots.cuda() + shift * page_size, freq.cuda(), big_k, big_v,
                                    **weights)
    assert torch.equal(large, small) and torch.equal(big_k[shift:], dk) and torch.equal(big_v[shift:], dv)


def test_two_calls_at_once_on_two_streams():
    cases = [_tree_case(73, [(5000, 40), (300, 8)], 32, 8, 128, 16, torch.bfloat16),
             _tree_case(74, [(64, 3)] * 40, 8, 2, 64, 16, torch.float16, chain=True)]
    want = [_run_tree(c) for c in cases]
    ds = [{k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()} for c in cases]
    ws = [pa.tree_attention_workspace(c["q"].shape[0], len(c["lpl"]), c["q"].shape[1], c["kp"].shape[2],
                                      c["q"].shape[2]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [pa.pa_v2_tree_attention(d["q"], d["kp"], d["vp"], d["idx"], d["indptr"], d["lpl"], d["fpo"], d["qo"],
                                       d["scale"], tree_mask=d["mask"], workspace=w, stream=s)
               for d, w, s in zip(ds, ws, streams)]
        torch.cuda.synchronize()
        for (out, lse), (ro, rl) in zip(got, want):
            assert torch.equal(out.cpu(), ro) and torch.equal(lse.cpu(), rl)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("graph", [False, True])
def test_a_whole_sliding_step(graph, tree):
    """Tables, q/k preparation and attention under a sliding window, eagerly and from a graph replayed with other
    lengths: each token's q and k at its own position, and its output over the rows that its own window holds."""
    dtype, hq, hkv, D, ps, B, window, cap_t, width, P = torch.bfloat16, 8, 2, 64, 16, 3, 50, 60, 30, 120
    rng, g = random.Random(91), torch.Generator().manual_seed(91)
    freq = torch.tensor([10000.0 ** (-j / 32) for j in range(32)], dtype=torch.float32)
    weights = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)]
    table = torch.randperm(P, generator=g)[:B * width].reshape(B, width).to(I32)
    kp, vp = (torch.randn(P, ps, hkv, D, generator=g).to(dtype) for _ in range(2))
    dtab, dk, dv, dfreq, dw = table.cuda(), kp.cuda(), vp.cuda(), freq.cuda(), [w.cuda() for w in weights]
    dc, dn, dpar = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda"), i32([-1] * cap_t).cuda()
    dx = torch.zeros(cap_t, hq + 2 * hkv, D, dtype=dtype, device="cuda")
    t, st = pa.StepTables.empty(B, B * width, cap_t, 1 if tree else 0), status_word()
    dq = torch.empty(cap_t, hq, D, dtype=dtype, device="cuda")
    out, lse = torch.empty_like(dq), torch.empty(cap_t, hq, device="cuda")
    ws = pa.tree_attention_workspace(cap_t, B, hq, hkv, D)

    def step():
        pa.pa_v2_build_tables(dc, dn, dtab, ps, t, parents=dpar if tree else None, sliding_window=window, status=st)
        pa.pa_v2_qk_rope_append(dx[:, :hq], dx[:, hq:hq + hkv], dx[:, hq + hkv:], t.positions, t.slots, dfreq, dk, dv,
                                q_out=dq, q_weight=dw[0], k_weight=dw[1], eps=1e-6, status=st)
        pa.pa_v2_tree_attention(dq, dk, dv, t.indices, t.indptr, t.last_page_len, t.first_page_offset, t.qo_indptr,
                                D ** -0.5, tree_mask=t.tree_mask, out=out, lse2_out=lse, workspace=ws, status=st,
                                sliding_window=window, positions=t.positions)

    replay = step
    if graph:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=s):
            step()
        replay = cg.replay
    for cached in ([200, 0, 37], [49, 50, 333]):
        fresh = [rng.randint(1, 19) for _ in range(B)]
        trees = [R.random_tree(rng, n) for n in fresh] if tree else [None] * B
        n = sum(fresh)
        x = torch.randn(n, hq + 2 * hkv, D, generator=g).to(dtype)
        dc.copy_(i32(cached))
        dn.copy_(i32(fresh))
        if tree:
            dpar[:n] = i32(p for ps_ in trees for p in ps_).cuda()
        dx[:n] = x.cuda()
        replay()
        torch.cuda.synchronize()
        assert int(st) == 0
        pos, own, seen = [], [], []
        for r, (c, m) in enumerate(zip(cached, fresh)):
            row = lambda at: int(table[r, at // ps]) * ps + at % ps
            for i in range(m):
                line = R.ancestors(trees[r], i)
                pos.append(c + len(line) - 1)
                own.append(row(c + i))
                seen.append([row(y) for y in range(max(pos[-1] - window + 1, 0), c)] +
                            [row(c + j) for j in reversed(line[:window])])
        q, k, v = dq[:n].cpu(), dk.cpu(), dv.cpu()
        for got, heads, w in ((q, x[:, :hq], weights[0]), (k.flatten(0, 1)[own], x[:, hq:hq + hkv], weights[1])):
            ref, mag = R.rope_ref(heads, w, 1e-6, pos, freq, False)
            assert ((got.double() - ref).abs() <= R.rope_tolerance(ref, mag, dtype)).all()
        assert torch.equal(v.flatten(0, 1)[own], x[:, hq + hkv:])
        ro, rl, to, tl = R.rows_attention_ref(q, k, v, seen, D ** -0.5)
        assert ((out[:n].cpu().double() - ro).abs() <= to).all() and ((lse[:n].cpu().double() - rl).abs() <= tl).all()
