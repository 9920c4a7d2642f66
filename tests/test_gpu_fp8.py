"""GPU: the 8-bit cache (pa_v2_qk_rope_append_fp8, pa_v2_attention_fp8) against plain 64-bit references, alone and
together."""
import math
import random

import pytest
import torch

import fp8_reference as F
import step_reference as R
from paged_attention_decode_gb300 import pa_v2 as pa

pytestmark = pytest.mark.gpu

I32 = torch.int32
E4M3 = F.E4M3
DT = [torch.float16, torch.bfloat16]


def i32(x):
    return torch.tensor(list(x), dtype=I32)


def status_word():
    return torch.zeros(1, dtype=I32, device="cuda")


def prefix(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _append_case(seed, reqs, page_size, hq, hkv, D, rot, dtype, norm, pad=0, size=1.7, packed=True, old=(-9, -4)):
    """reqs: (cached, new) per request.  Pages are dealt out at random; what lies on them is random codes."""
    g = torch.Generator().manual_seed(seed)
    counts = [(c + n - 1) // page_size - c // page_size + 1 if n else 0 for c, n in reqs]
    P = sum(counts) + 3
    ids = torch.randperm(P, generator=g).tolist()
    slots, positions, base = [], [], 0
    for (c, n), k in zip(reqs, counts):
        slots += [ids[base + x // page_size - c // page_size] * page_size + x % page_size for x in range(c, c + n)]
        positions += range(c, c + n)
        base += k
    T = len(slots) + pad
    if packed:
        x = (torch.randn(T, hq + 2 * hkv, D, generator=g) * size).to(dtype)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = ((torch.randn(T, h, D, generator=g) * size).to(dtype) for h in (hq, hkv, hkv))
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype) if norm else None for _ in range(2)]

    def pool():
        codes = (torch.randn(P, page_size, hkv, D, generator=g) * 90).clamp(-448, 448).to(E4M3)
        return codes, torch.randint(old[0], old[1] + 1, (P, hkv), generator=g).to(torch.int8)

    kp, ke = pool()
    vp, ve = pool()
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float32) / max(1, rot // 2)) if rot else None
    return dict(q=q, k=k, v=v, qw=w[0], kw=w[1], pos=i32(positions + [0] * pad), slots=i32(slots + [-1] * pad),
                kp=kp, vp=vp, ke=ke, ve=ve, freq=freq, eps=1e-5)


def _to(x, stream=None):
    return None if x is None else x.cuda()


def _packed_cuda(c):
    """q, k and v on the GPU as views of one tensor where they are views of one."""
    if c["q"].is_contiguous():
        return c["q"].cuda(), c["k"].cuda(), c["v"].cuda()
    hq, hkv = c["q"].shape[1], c["k"].shape[1]
    x = torch.cat((c["q"], c["k"], c["v"]), 1).cuda()
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def _run_append(c, interleaved=False, q_dtype=None, status=None, stream=None, cache=None, q_out=None):
    q, k, v = _packed_cuda(c)
    cache = cache or [c[n].cuda() for n in ("kp", "vp", "ke", "ve")]
    out = pa.pa_v2_qk_rope_append_fp8(q, k, v, c["pos"].cuda(), c["slots"].cuda(), _to(c["freq"]), *cache,
                                      q_out=q_out, q_weight=_to(c["qw"]), k_weight=_to(c["kw"]), eps=c["eps"],
                                      interleaved=interleaved, q_dtype=q_dtype, status=status, stream=stream)
    torch.cuda.synchronize()
    return out, cache


def _check_append(c, out, cache, interleaved=False):
    freq = c["freq"] if c["freq"] is not None else []
    live = (c["slots"] >= 0) & (c["slots"] < c["kp"].shape[0] * c["kp"].shape[1])
    rq, mq = R.rope_ref(c["q"], c["qw"], c["eps"], c["pos"], freq, interleaved)
    got = out.cpu().double()
    # rope_tolerance's half step is of normal numbers; below them a step is eps times the smallest normal one (f16: 2^-24),
    # and an element that is not rotated has no larger partner whose size would cover it
    fi = torch.finfo(out.dtype)
    fine = rq.isfinite()                       # (an infinity or NaN of q is compared as it is)
    bad = live[:, None, None] & ~fine
    assert torch.equal(got[bad].nan_to_num(3.0), rq[bad].nan_to_num(3.0))
    fine = live[:, None, None] & fine
    off = (got - rq).abs() - R.rope_tolerance(rq, mq, out.dtype) - fi.eps / 2 * fi.smallest_normal
    assert (off[fine] <= 0).all(), (float(off[fine].max()), rq[fine][off[fine] > 0][:5], got[fine][off[fine] > 0][:5])
    rk, mk = R.rope_ref(c["k"], c["kw"], c["eps"], c["pos"], freq, interleaved)
    v = c["v"].double()
    for x, mag, pool, exps, new, new_exps in ((rk, mk, c["kp"], c["ke"], cache[0], cache[2]),
                                              (v, torch.zeros_like(v), c["vp"], c["ve"], cache[1], cache[3])):
        low, high, want = F.append_ref(x, mag, pool, exps, c["slots"], new_exps.cpu())
        assert torch.equal(new_exps.cpu().long(), want)
        y = new.cpu().float().double()
        assert torch.equal(y.isnan(), low.isnan())
        assert ((y >= low) & (y <= high) | y.isnan()).all()
        # what is not of the call keeps its bits
        ps = pool.shape[1]
        pages = torch.unique(c["slots"][live].long() // ps)
        rest = torch.ones(pool.shape[0], dtype=torch.bool)
        rest[pages] = False
        assert torch.equal(new.cpu().view(torch.uint8)[rest], pool.view(torch.uint8)[rest])


@pytest.mark.parametrize("dtype,q_dtype", [(torch.float16, None), (torch.float16, torch.float32), (torch.bfloat16, None),
                                           (torch.bfloat16, torch.float32), (torch.float32, None)])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 32, False), (64, 64, False),
                                               (64, 48, True), (128, 0, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_matches_the_definition(dtype, q_dtype, D, rot, interleaved, norm):
    c = _append_case(7, [(0, 21), (5, 1), (30, 40), (16, 0), (15, 2)], 16, 12, 4, D, rot, dtype, norm, pad=3)
    st = status_word()
    out, cache = _run_append(c, interleaved, q_dtype, st)
    assert int(st) == 0 and out.dtype == (q_dtype or dtype)
    _check_append(c, out, cache, interleaved)


@pytest.mark.parametrize("page_size", [1, 2, 5, 7, 16, 32, 48, 64, 100, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_page_sizes_and_runs(page_size, dtype):
    # runs of one token, within a page, to its end, whole pages, more than a warp holds, and the rest of one
    reqs = [(0, 1), (page_size // 2, 1), (page_size // 2, page_size), (0, 2 * page_size + 1), (3, 300), (1000001, 9)]
    c = _append_case(page_size, reqs, page_size, 6, 3, 64 if page_size % 2 else 128, 64, dtype, True)
    out, cache = _run_append(c)
    _check_append(c, out, cache)


@pytest.mark.parametrize("hq,hkv,packed", [(1, 1, True), (32, 8, True), (28, 4, False), (7, 7, True), (40, 20, False)])
@pytest.mark.parametrize("T", [1, 17, 700])
def test_append_head_counts_lengths_and_strides(hq, hkv, packed, T):
    c = _append_case(T + hq, [(11, T)], 16, hq, hkv, 128, 128, torch.bfloat16, True, packed=packed)
    out, cache = _run_append(c)
    _check_append(c, out, cache)


def test_append_many_requests_of_one_token():
    rng = random.Random(3)
    c = _append_case(3, [(rng.randint(0, 5000), 1) for _ in range(1500)], 16, 4, 2, 64, 64, torch.float16, False)
    out, cache = _run_append(c)
    _check_append(c, out, cache)


def test_append_an_exponent_grows_never_falls_and_begins_anew():
    ps, hkv, D = 4, 1, 64
    # pages: grows by 9, stays, begins anew below a huge old exponent, begins anew from nothing, an exponent out of range
    slots = [0 * ps + 2, 1 * ps + 3, 2 * ps, 3 * ps, 4 * ps + 1, 5 * ps + 1]
    old = torch.tensor([[-9], [3], [7], [-15], [100], [-100]], dtype=torch.int8)
    v = torch.zeros(6, 1, D)
    for t, top in enumerate((448.0, 1.0, 0.5, 0.0, 2.0, 3.0)):
        v[t, 0, t] = -top
        v[t, 0, 40 + t] = top / 7
    codes = torch.arange(256, dtype=torch.uint8)[(torch.arange(256) & 0x7f) != 0x7f][:192].view(E4M3)
    pool = codes.repeat(8)[:6 * ps * D].reshape(6, ps, hkv, D)
    c = dict(q=v, k=v, v=v, qw=None, kw=None, pos=i32([0] * 6), slots=i32(slots), kp=pool, vp=pool.clone(), ke=old,
             ve=old.clone(), freq=None, eps=0.0)
    out, cache = _run_append(c)
    _check_append(c, out, cache)
    assert cache[3].flatten().tolist() == [0, 3, F.need_of(0.5), -15, 7, F.need_of(3.0)]
    # the same call again changes nothing more
    before = [x.clone() for x in cache]
    _run_append(c, cache=cache)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, cache))


def test_append_every_code_rescaled_by_every_step():
    """A page's earlier codes, all of them, through each growth of its exponent."""
    ps, D = 5, 64
    codes = torch.arange(256, dtype=torch.uint8).reshape(4, D)
    pool = torch.zeros(22, ps, 1, D, dtype=torch.uint8)
    pool[:, :4, 0] = codes
    pool = pool.view(E4M3)
    v = torch.zeros(22, 1, D)
    for d in range(1, 23):
        v[d - 1, 0, 3] = 448.0 * 2.0 ** (-15 + d)
    c = dict(q=v, k=v, v=v, qw=None, kw=None, pos=i32([0] * 22), slots=i32(p * ps + 4 for p in range(22)), kp=pool,
             vp=pool.clone(), ke=torch.full((22, 1), -15, dtype=torch.int8), ve=torch.full((22, 1), -15, dtype=torch.int8),
             freq=None, eps=0.0)
    out, cache = _run_append(c)
    assert cache[2].flatten().tolist() == list(range(-14, 8))
    for d in range(1, 23):
        old = codes.view(E4M3).float().double()
        want = F.code_of(old * 2.0 ** -d)
        got = cache[0][d - 1, :4, 0].cpu().float().double()
        assert torch.equal(got.nan_to_num(999.0), want.nan_to_num(999.0)), d


def test_append_saturates_and_keeps_nan_and_infinity_as_nan():
    D = 64
    v = torch.randn(4, 2, D, generator=torch.Generator().manual_seed(1))
    v[0, 0, 5], v[0, 1, 6] = math.inf, math.nan            # beside values of ordinary size, which set the exponent
    v[1, 0], v[1, 1] = math.nan, -math.inf                 # nothing finite
    v[2, 0, 0], v[2, 1, 1] = 1e30, -60000.0                # above what the range holds
    v[3, 0, 0] = -57344.0
    z = torch.zeros(4, 8, 2, D, dtype=torch.uint8).view(E4M3)
    e = torch.zeros(4, 2, dtype=torch.int8)
    c = dict(q=v, k=v, v=v, qw=None, kw=None, pos=i32([3] * 4), slots=i32([0, 8, 16, 24]), kp=z, vp=z.clone(), ke=e,
             ve=e.clone(), freq=None, eps=0.0)
    out, cache = _run_append(c)
    _check_append(c, out, cache)
    got = cache[1].cpu().float()
    assert got[0, 0, 0, 5].isnan() and got[0, 0, 1, 6].isnan() and got[0, 0].isnan().sum() == 2
    assert got[1, 0].isnan().all() and cache[3][1].tolist() == [-15, -15]
    assert float(got[2, 0, 0, 0]) == 448.0 and float(got[2, 0, 1, 1]) == -448.0 and cache[3][2].tolist() == [7, 7]
    assert float(got[3, 0, 0, 0]) == -448.0 and int(cache[3][3, 0]) == 7


def test_append_padding_and_bad_slots_are_skipped():
    c = _append_case(9, [(3, 6), (20, 2)], 16, 4, 2, 64, 64, torch.float16, True, pad=2)
    rows = c["kp"].shape[0] * 16
    c["slots"] = torch.cat((c["slots"][:6], i32([rows, 2 ** 31 - 1, -5, -2 ** 31])))
    st = status_word()
    q_out = torch.full((10, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    out, cache = _run_append(c, status=st, q_out=q_out)
    assert int(st) == pa.DEVICE_BAD_SLOT
    assert (out[6:] == 9.0).all()
    _check_append(c, out, cache)


def _refused(slots, rows, page_size):
    """Which tokens skipped ones cut off from an earlier token of their page."""
    out, before, last = [], False, -1          # of the nearest earlier token that is not skipped: refused, its number
    for t, s in enumerate(slots.tolist()):
        out.append(False)
        if 0 <= s < rows:
            same = last >= 0 and int(slots[last]) // page_size == s // page_size
            out[-1] = before = same and (before or t > last + 1)
            last = t
    return torch.tensor(out)


def _check_append_refusing(c, **kw):
    """A call whose skipped tokens split pages: what is cut off is not stored and recorded, all else is as without it."""
    ps = c["kp"].shape[1]
    rows = c["kp"].shape[0] * ps
    cut = _refused(c["slots"], rows, ps)
    st = status_word()
    out, cache = _run_append(c, status=st, **kw)
    assert int(st) == (pa.DEVICE_BAD_SLOT if cut.any() or (c["slots"] >= rows).any() else 0)
    _check_append(dict(c, slots=torch.where(cut, -1, c["slots"])), out, cache)
    want, mag = R.rope_ref(c["q"][cut], c["qw"], c["eps"], c["pos"][cut], c["freq"], False)
    got = out.cpu().double()[cut]
    fi = torch.finfo(out.dtype)
    assert ((got - want).abs() <= R.rope_tolerance(want, mag, out.dtype) + fi.eps / 2 * fi.smallest_normal).all()
    return cut


@pytest.mark.parametrize("gap", [1, 2, 31, 32, 33, 70, 500])
@pytest.mark.parametrize("skipped", [-1, -2 ** 31, 2 ** 31 - 1])
def test_append_skipped_tokens_between_tokens_of_a_page(gap, skipped):
    """Two tokens of a page, skipped ones, two more: the page's first run alone is stored, whatever lies between."""
    c = _append_case(9, [(3, 2 + gap + 2), (40, 3)], 1024 // 4, 4, 2, 64, 64, torch.float16, True)
    c["slots"][2:2 + gap] = skipped
    if 2 + gap + 2 > 253:
        c["slots"][2 + gap:4 + gap] = c["slots"][:2] + 10       # (of the same page, which ends before them)
    cut = _check_append_refusing(c)
    assert cut.nonzero().flatten().tolist() == [2 + gap, 3 + gap]


@pytest.mark.parametrize("page_size", [1, 2, 5, 16, 64, 256])
@pytest.mark.parametrize("T,share", [(40, 0.2), (700, 0.1), (700, 0.9), (1200, 0.3)])
def test_append_skipped_tokens_anywhere(page_size, T, share):
    """Long calls, stretches of one token and of more, random tokens of every page skipped, as padding or past the pool."""
    g = torch.Generator().manual_seed(T + page_size)
    c = _append_case(T, [(5, T // 2), (page_size // 2, T - T // 2)], page_size, 4, 2, 64, 16, torch.bfloat16, False)
    rows = c["kp"].shape[0] * page_size
    drop, past = torch.rand(T, generator=g) < share, torch.rand(T, generator=g) < 0.3
    c["slots"] = torch.where(drop, torch.where(past, rows + 3, -1), c["slots"]).to(I32)
    cut = _check_append_refusing(c)
    assert cut.any() == (page_size > 2)


@pytest.mark.parametrize("width", [1, 7, 33, 100])
def test_append_requests_padded_to_one_width(width):
    """A row of `width` tokens a request, the last ones padding: nothing is cut off."""
    lens = [1, width, max(1, width // 2), 0, width, 1]
    c = _append_case(width, [(7 * r, n) for r, n in enumerate(lens)], 16, 4, 2, 64, 64, torch.float16, True)
    parts = torch.split(torch.arange(sum(lens)), lens)
    at = torch.cat([torch.cat((p, torch.zeros(width - len(p), dtype=torch.long))) for p in parts])
    live = torch.cat([torch.arange(width) < n for n in lens])
    for n in ("q", "k", "v", "pos", "slots"):
        c[n] = c[n][at]
    c["slots"] = torch.where(live, c["slots"], -1).to(I32)
    assert not _check_append_refusing(c).any()


def test_append_tokens_of_a_page_in_any_order():
    c = _append_case(4, [(2, 30)], 16, 4, 2, 64, 64, torch.bfloat16, True)
    perm = torch.tensor([5, 3, 13, 0, 1, 2, 4, 6, 7, 8, 9, 10, 11, 12] + [29 - i for i in range(16)])
    for n in ("q", "k", "v", "pos", "slots"):
        c[n] = c[n][perm]
    out, cache = _run_append(c)
    _check_append(c, out, cache)


def test_append_one_token_at_a_time_equals_a_growing_page():
    """Tokens appended in separate calls: each value lies within its last rounding and one more for each growth."""
    g = torch.Generator().manual_seed(8)
    T, D = 40, 128
    v = (torch.randn(T, 1, D, generator=g) * torch.exp2(torch.linspace(-6, 6, T))[:, None, None]).half()
    z = torch.zeros(4, 16, 1, D, dtype=torch.uint8).view(E4M3)
    e = torch.zeros(4, 1, dtype=torch.int8)
    cache = [z.cuda(), z.cuda(), e.cuda(), e.cuda()]
    pool, exps = z, e
    for t in range(T):
        c = dict(q=v[t:t + 1], k=v[t:t + 1], v=v[t:t + 1], qw=None, kw=None, pos=i32([t]), slots=i32([t]), kp=z, vp=z,
                 ke=e, ve=e, freq=None, eps=0.0)
        _run_append(c, cache=cache)
        x = v[t:t + 1].double()
        low, high, exps = F.append_ref(x, torch.zeros_like(x), pool, exps, c["slots"])
        assert torch.equal(low, high)
        pool = low.float().to(E4M3)
    assert torch.equal(cache[1].cpu().view(torch.uint8), pool.view(torch.uint8)) and torch.equal(cache[3].cpu().long(), exps)
    assert torch.equal(cache[0].view(torch.uint8), cache[1].view(torch.uint8))


def test_append_empty_call_in_a_graph_and_on_another_stream():
    c = _append_case(5, [(7, 30), (0, 3)], 16, 8, 2, 128, 128, torch.bfloat16, True)
    out, cache = _run_append(c)
    first = [out.clone(), *[x.clone() for x in cache]]
    q, k, v = _packed_cuda(c)
    none = pa.pa_v2_qk_rope_append_fp8(q[:0], k[:0], v[:0], c["pos"][:0].cuda(), c["slots"][:0].cuda(), c["freq"].cuda(),
                                       *cache)
    assert none.shape == (0, 8, 128)
    args = (q, k, v, c["pos"].cuda(), c["slots"].cuda(), c["freq"].cuda())
    kw = dict(q_weight=c["qw"].cuda(), k_weight=c["kw"].cuda(), eps=c["eps"])
    cache = [c[n].cuda() for n in ("kp", "vp", "ke", "ve")]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = pa.pa_v2_qk_rope_append_fp8(*args, *cache, stream=s, **kw)
    s.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, [out, *cache]))
    cache = [c[n].cuda() for n in ("kp", "vp", "ke", "ve")]
    graph, q_out = torch.cuda.CUDAGraph(), torch.zeros_like(out)
    with torch.cuda.graph(graph):
        pa.pa_v2_qk_rope_append_fp8(*args, *cache, q_out=q_out, **kw)
    for x, n in zip(cache, ("kp", "vp", "ke", "ve")):
        x.copy_(c[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, [q_out, *cache]))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _attn_case(seed, reqs, hq, hkv, D, page_size, dtype, window=0, sinks=0, trees=None, words=None, fpos=None, slack=3,
               give_back=False):
    """reqs: (cached, new) per request; fpos: the first listed entry of each; trees: parents per request."""
    g = torch.Generator().manual_seed(seed)
    fpos = fpos or [0] * len(reqs)
    counts = [-(-(f + c + n) // page_size) for (c, n), f in zip(reqs, fpos)]
    P = sum(counts) + slack
    ids = torch.randperm(P, generator=g)[:sum(counts)].to(I32)
    T = sum(n for _, n in reqs)

    def pool():
        codes = (torch.randn(P, page_size, hkv, D, generator=g) * 64).clamp(-448, 448).to(E4M3)
        return codes, torch.randint(-8, -3, (P, hkv), generator=g).to(torch.int8)

    kp, ke = pool()
    vp, ve = pool()
    indptr = prefix(counts)
    seen, positions = [], []
    for r, ((c, n), f) in enumerate(zip(reqs, fpos)):
        for i in range(n):
            line = R.ancestors(trees[r], i) if trees else None
            depth = len(line) - 1 if trees else i
            if trees and window:
                line = line[:window]
            seen.append(F.seen_rows(ids[indptr[r]:indptr[r + 1]], page_size, f, c + n, n, i, window, sinks,
                                    None if line is None else set(line), depth))
            positions.append(c + depth)
    mask = None
    if trees:
        words = words or max(1, -(-max(n for _, n in reqs) // 32))
        rows = []
        for parents in trees:
            for i in range(len(parents)):
                line = R.ancestors(parents, i)[:window or None]
                rows.append(R.words_of(sum(1 << j for j in line), words))
        mask = torch.tensor(rows, dtype=I32).reshape(T, words)
    if give_back:            # pages that nobody sees: gone
        used = {row // page_size for rows in seen for row in rows}
        for s in range(len(ids)):
            if int(ids[s]) not in used:
                ids[s] = -1
    total = [f + c + n for (c, n), f in zip(reqs, fpos)]
    return dict(q=(1.3 * torch.randn(T, hq, D, generator=g)).to(dtype), kp=kp, vp=vp, ke=ke, ve=ve, ids=ids,
                indptr=i32(indptr), lpl=i32((t - 1) % page_size + 1 if t else 0 for t in total), fpo=i32(fpos),
                qo=i32(prefix(n for _, n in reqs)), mask=mask, pos=i32(positions), window=window, sinks=sinks,
                scale=D ** -0.5, seen=seen)


def _run_attn(c, pad=0, **kw):
    q = c["q"] if not pad else torch.cat((c["q"], torch.zeros(pad, *c["q"].shape[1:], dtype=c["q"].dtype)))
    mask, pos = c["mask"], c["pos"]
    if pad:
        pos = torch.cat((pos, torch.zeros(pad, dtype=I32)))
        mask = None if mask is None else torch.cat((mask, torch.zeros(pad, mask.shape[1], dtype=I32)))
    out, lse = pa.pa_v2_attention_fp8(
        q.cuda(), c["kp"].cuda(), c["vp"].cuda(), c["ke"].cuda(), c["ve"].cuda(), c["ids"].cuda(), c["indptr"].cuda(),
        c["lpl"].cuda(), c["fpo"].cuda(), c["qo"].cuda(), c["scale"], tree_mask=_to(mask), positions=pos.cuda(),
        sliding_window=c["window"], sinks=c["sinks"], **kw)
    torch.cuda.synchronize()
    return out, lse


def _attn_ref(c):
    return F.attention_ref(c["q"], F.values(c["kp"], c["ke"]), F.values(c["vp"], c["ve"]), c["seen"], c["scale"])


def _close(got, ref):
    out, lse = (x.cpu().double() for x in got)
    ro, rl, to, tl = ref
    n = len(ro)
    assert torch.equal(lse[:n] == -math.inf, rl == -math.inf)
    fine = rl > -math.inf
    assert ((out[:n] - ro).abs() <= to).all(), float(((out[:n] - ro).abs() - to).max())
    assert ((lse[:n] - rl).abs() <= tl)[fine].all(), float((lse[:n] - rl)[fine].abs().max())


def _check_attn(c, **kw):
    st = status_word()
    got = _run_attn(c, status=st, **kw)
    assert int(st) == 0
    _close(got, _attn_ref(c))
    return got


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("reqs", [[(0, 1)], [(1, 1)], [(30, 1)], [(31, 1)], [(32, 1)], [(255, 1)], [(1000, 1)],
                                  [(0, 2)], [(0, 7)], [(29, 3)], [(100, 5), (0, 1), (64, 3)], [(0, 0), (33, 2), (5, 0)]])
def test_attention_lengths(reqs, D, dtype):
    _check_attn(_attn_case(1, reqs, 8, 2, D, 16, dtype))


@pytest.mark.parametrize("page_size", [1, 2, 3, 5, 7, 8, 12, 15, 16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mid", [False, True])
def test_attention_page_sizes_and_first_offsets(page_size, D, mid):
    reqs = [(517, 1), (3, 2), (77, 3)]
    fpos = [page_size - 1, page_size // 2, 1 % page_size] if mid else None
    _check_attn(_attn_case(page_size, reqs, 4, 2, D, page_size, torch.float16, fpos=fpos))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (8, 8), (12, 4), (16, 1), (40, 8), (33, 1), (64, 2)])
@pytest.mark.parametrize("n", [1, 3])
def test_attention_head_groups(hq, hkv, n):
    _check_attn(_attn_case(hq, [(200, n), (40, n)], hq, hkv, 128, 16, torch.bfloat16))


@pytest.mark.parametrize("n,tree", [(9, False), (33, False), (33, True), (65, True), (130, False), (200, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_new_tokens(n, tree, D):
    rng = random.Random(n)
    trees = [R.random_tree(rng, n), R.random_tree(rng, 4)] if tree else None
    _check_attn(_attn_case(n, [(61, n), (9, 4)], 4, 2, D, 16, torch.float16, trees=trees))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("reqs,hq,hkv", [([(20000, 1)], 8, 2), ([(20000, 1)], 4, 1), ([(9000, 2), (1, 1)], 8, 1),
                                         ([(6000, 9)], 4, 1)])
def test_attention_long_contexts_split_over_the_machine(reqs, hq, hkv, dtype):
    _check_attn(_attn_case(5, reqs, hq, hkv, 128, 16, dtype))


def test_attention_many_ragged_requests():
    rng = random.Random(2)
    reqs = [(rng.choice([0, 5, 31, 32, rng.randint(0, 700)]), rng.choice([0, 1, 1, 2])) for _ in range(90)]
    _check_attn(_attn_case(2, reqs, 8, 2, 64, 16, torch.bfloat16))


def test_attention_more_requests_than_threads():
    rng = random.Random(4)
    reqs = [(rng.randint(0, 40), rng.choice([0, 1, 1, 1])) for _ in range(700)]
    _check_attn(_attn_case(4, reqs, 4, 2, 64, 5, torch.float16))


WINDOWS = [([(300, 1)], 64, 4), ([(300, 1)], 64, 0), ([(300, 1)], 1, 1), ([(300, 1)], 1000, 7), ([(40, 1), (3, 1), (0, 1)], 16, 33),
           ([(300, 6), (10, 6), (0, 6)], 40, 3), ([(300, 9)], 4, 2), ([(200, 70)], 16, 5), ([(5000, 1), (900, 2)], 129, 100),
           ([(64, 1), (65, 1), (95, 1), (96, 1)], 32, 32)]


@pytest.mark.parametrize("reqs,window,sinks", WINDOWS)
@pytest.mark.parametrize("page_size,D", [(16, 128), (5, 64), (64, 64), (1, 128)])
def test_attention_windows_and_sinks(reqs, window, sinks, page_size, D):
    _check_attn(_attn_case(window + sinks, reqs, 8, 2, D, page_size, torch.float16, window, sinks, give_back=True))


@pytest.mark.parametrize("window,sinks", [(0, 0), (12, 3), (70, 0), (3, 40)])
def test_attention_trees_under_windows(window, sinks):
    rng = random.Random(window)
    reqs = [(150, 40), (2, 33), (0, 9), (77, 1)]
    trees = [R.random_tree(rng, n) for _, n in reqs]
    _check_attn(_attn_case(7, reqs, 6, 2, 128, 16, torch.bfloat16, window, sinks, trees=trees, give_back=True))


def test_attention_sinks_that_new_tokens_are():
    # a short request whose new tokens lie among the first `sinks`, with a window shorter than them
    _check_attn(_attn_case(3, [(2, 12), (0, 20)], 4, 2, 64, 16, torch.float16, 3, 9))


def test_attention_padded_rows_are_left_alone():
    c = _attn_case(6, [(100, 2), (31, 1)], 8, 2, 128, 16, torch.float16)
    out = torch.full((7, 8, 128), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((7, 8), 6.0, device="cuda")
    got = _run_attn(c, pad=4, out=out, lse2_out=lse)
    _close(got, _attn_ref(c))
    assert (out[3:] == 5.0).all() and (lse[3:] == 6.0).all()


def test_attention_masks_that_leave_rows_empty():
    c = _attn_case(8, [(0, 5), (40, 5)], 4, 2, 64, 16, torch.float16, trees=[[-1, 0, 1, -1, 3]] * 2)
    c["mask"][1], c["mask"][3] = 0, 0
    c["seen"][1], c["seen"][3] = [], []
    out, lse = _check_attn(c)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("page_size,D", [(16, 128), (5, 128), (64, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_attention_nothing_hidden_reaches_a_result(page_size, D, window, sinks):
    """NaN codes everywhere that no token sees, and in rows that some tokens do not see."""
    rng = random.Random(1)
    reqs = [(70, 7), (9, 3), (200, 1)]
    trees = [R.random_tree(rng, n) for _, n in reqs]
    c = _attn_case(11, reqs, 4, 2, D, page_size, torch.float16, window, sinks, trees=trees)
    ref = _attn_ref(c)
    seen = torch.zeros(c["kp"].shape[0] * page_size, dtype=torch.bool)
    for rows in c["seen"]:
        seen[rows] = True
    for n in ("kp", "vp"):
        c[n].view(torch.uint8).flatten(0, 1)[~seen] = 0x7f
    st = status_word()
    _close(_run_attn(c, status=st), ref)
    assert int(st) == 0


@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("hq,n", [(8, 1), (8, 12), (4, 40)])
def test_attention_nan_reaches_the_rows_that_see_it_and_no_other(page_size, hq, n):
    rng = random.Random(n)
    reqs = [(100, n), (40, n)]
    c = _attn_case(13, reqs, hq, 2, 128, page_size, torch.bfloat16, 30, 2,
                   trees=[R.random_tree(rng, n, 0.3) for _ in reqs])
    hit = sorted({rows[k] for rows in c["seen"] for k in (0, len(rows) // 2, -1)})
    vals = c["vp"].view(torch.uint8).flatten(0, 1)
    for j, row in enumerate(hit):
        vals[row, j % 2, (7 * j) % 128] = 0x7f if j % 3 else 0xff
    got = _run_attn(c)
    clean = dict(c, vp=c["vp"].float().nan_to_num(0.0).to(E4M3))
    ro, rl, to, tl = _attn_ref(clean)
    nan = torch.zeros(ro.shape, dtype=torch.bool)
    flat = c["vp"].float().isnan().flatten(0, 1)
    for t, rows in enumerate(c["seen"]):
        nan[t] = flat[rows].any(0).repeat_interleave(hq // 2, 0)
    assert nan.any() and not nan.all()
    out = got[0].cpu().double()
    assert torch.equal(out.isnan(), nan)
    assert ((out - ro).abs() <= to)[~nan].all() and ((got[1].cpu().double() - rl).abs() <= tl).all()
    # a NaN key makes its rows' results NaN
    c = dict(clean, kp=c["kp"].clone())
    c["kp"].view(torch.uint8).flatten(0, 1)[hit[0], 0, 3] = 0x7f
    out, lse = (x.cpu() for x in _run_attn(c))
    for t, rows in enumerate(c["seen"]):
        assert out[t, :hq // 2].isnan().all() == (hit[0] in rows) and out[t, hq // 2:].isfinite().all()
        assert lse[t, :hq // 2].isnan().all() == (hit[0] in rows)


@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 2)])
@pytest.mark.parametrize("hq,n", [(8, 1), (8, 4), (8, 12), (4, 40), (8, 60)])
def test_attention_a_nan_key_reaches_all_of_the_rows_that_see_it_and_nothing_else(page_size, window, sinks, hq, n):
    """Every element of the rows that see it, and not one of the others, whose results are those without it."""
    rng = random.Random(n)
    reqs = [(100, n), (40, n)]
    c = _attn_case(14, reqs, hq, 2, 128, page_size, torch.bfloat16, window, sinks,
                   trees=[R.random_tree(rng, n, 0.3) for _ in reqs])
    ro, rl, to, tl = _attn_ref(c)
    for hit in sorted({rows[k] for rows in c["seen"][::max(1, n // 3)] for k in (0, len(rows) // 2, -1)}):
        d = dict(c, kp=c["kp"].clone())
        d["kp"].view(torch.uint8).flatten(0, 1)[hit, 1, 77] = 0xff
        out, lse = (x.cpu().double() for x in _run_attn(d))
        nan = torch.zeros(ro.shape, dtype=torch.bool)
        for t, rows in enumerate(c["seen"]):
            nan[t, hq // 2:] = hit in rows
        assert nan.any() and not nan.all() and torch.equal(out.isnan(), nan) and torch.equal(lse.isnan(), nan[..., 0])
        assert ((out - ro).abs() <= to)[~nan].all() and ((lse - rl).abs() <= tl)[~nan[..., 0]].all()


# -- blocks of 24 rows: 33 to 72 query rows per KV head (or 17 to 24) where a warp meets many keys, or a list could hold them

def _listed_more(c, hkv, page_size):
    """The same with a longer index array: more than four tiles of 32 keys for each of eight warps of up to 160 SMs."""
    pad = 4 * 32 * 8 * 160 // hkv // page_size + 1
    return dict(c, ids=torch.cat((c["ids"], torch.zeros(pad, dtype=I32))))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("page_size,D", [(16, 128), (5, 64), (64, 64), (1, 128), (7, 128)])
@pytest.mark.parametrize("reqs", [[(517, 9), (3, 10), (77, 15), (0, 0), (33, 16)], [(900, 5)], [(40, 14), (0, 13)]])
def test_attention_blocks_of_24_rows(reqs, page_size, D, tree):
    rng = random.Random(D)
    trees = [R.random_tree(rng, n) for _, n in reqs] if tree else None
    c = _attn_case(21, reqs, 8, 2, D, page_size, torch.bfloat16 if tree else torch.float16, trees=trees)
    _check_attn(_listed_more(c, 2, page_size))


@pytest.mark.parametrize("page_size,D", [(16, 64), (5, 64), (16, 128)])
@pytest.mark.parametrize("window,sinks,tree", [(200, 5, False), (210, 0, False), (190, 20, True)])
def test_attention_blocks_of_24_rows_under_windows(window, sinks, tree, page_size, D):
    rng = random.Random(window)
    reqs = [(rng.choice([0, 3, 190, 200, 333, 700]), rng.choice([1, 5, 9])) for _ in range(30)]
    reqs[3], reqs[7] = (205, 5), (700, 6)
    trees = [R.random_tree(rng, n, 0.3) for _, n in reqs] if tree else None
    group = max(g for g in (4, 5, 6) if 17 <= -(-sum(n for _, n in reqs) // 30) * g <= 24)
    c = _attn_case(22, reqs, 32 * group, 32, D, page_size, torch.float16, window, sinks, trees=trees, give_back=True)
    _check_attn(_listed_more(c, 32, page_size))


@pytest.mark.parametrize("page_size", [16, 5])
def test_attention_blocks_of_24_rows_nan_only_where_it_is_seen(page_size):
    rng = random.Random(3)
    reqs = [(100, 12), (40, 11)]
    c = _attn_case(23, reqs, 8, 2, 128, page_size, torch.bfloat16, trees=[R.random_tree(rng, n, 0.3) for _, n in reqs])
    hit = sorted({rows[k] for rows in c["seen"] for k in (0, len(rows) // 2, -1)})[1:]  # (in new tokens that some see)
    shown = set.intersection(*map(set, c["seen"][:12])) | set.intersection(*map(set, c["seen"][12:]))
    hit = [row for row in hit if row not in shown]
    for j, row in enumerate(hit):
        c["vp"].view(torch.uint8).flatten(0, 1)[row, j % 2, (7 * j) % 128] = 0x7f if j % 3 else 0xff
    out = _run_attn(_listed_more(c, 2, page_size))[0].cpu().double()
    flat = c["vp"].float().isnan().flatten(0, 1)
    nan = torch.stack([flat[rows].any(0).repeat_interleave(4, 0) for rows in c["seen"]])
    assert nan.any() and not nan.all() and torch.equal(out.isnan(), nan)
    ro, _, to, _ = _attn_ref(dict(c, vp=c["vp"].float().nan_to_num(0.0).to(E4M3)))
    assert ((out - ro).abs() <= to)[~nan].all()


# -- more than 96 query rows per KV head: pages written out in q's type, the tree attention over them

MANY = [([(300, 60)], 8, 2, 0, 0), ([(0, 130)], 4, 2, 0, 0), ([(500, 70), (33, 50), (7, 0), (0, 61)], 8, 2, 0, 0),
        ([(900, 60), (20, 60)], 8, 2, 100, 5), ([(900, 60), (3, 60)], 8, 2, 30, 0), ([(400, 200)], 4, 4, 16, 40)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("reqs,hq,hkv,window,sinks", MANY)
@pytest.mark.parametrize("page_size,D,tree", [(16, 128, False), (5, 64, False), (16, 64, True), (256, 128, True), (1, 128, False)])
def test_attention_many_rows(reqs, hq, hkv, window, sinks, page_size, D, tree, dtype):
    rng = random.Random(window)
    trees = [R.random_tree(rng, n) for _, n in reqs] if tree else None
    _check_attn(_attn_case(61 + window, reqs, hq, hkv, D, page_size, dtype, window, sinks, trees=trees, give_back=True))


@pytest.mark.parametrize("page_size,D", [(16, 128), (5, 64), (64, 64), (256, 128)])
@pytest.mark.parametrize("window", [0, 33])
def test_attention_many_rows_from_a_first_offset(page_size, D, window):
    """Lists that begin inside a page, as a trimmed table's do, whole or with a window that hides their first rows."""
    reqs, fpos = [(300, 60), (2, 70), (700, 50)], [page_size - 1, page_size // 2, 1 % page_size]
    c = _attn_case(62, reqs, 8, 2, D, page_size, torch.bfloat16, window, fpos=fpos, give_back=True)
    _check_attn(c)


@pytest.mark.parametrize("window", [40, 300])
@pytest.mark.parametrize("tree", [False, True])
def test_sliding_tables_feed_the_attention_of_many_rows(window, tree):
    """pa_v2_build_tables_sliding's tables of a prompt's chunks and of wide trees, beside a request without tokens."""
    rng = random.Random(window)
    cached, new, ps, hq, hkv, D, width = [700, 33, 0, 90], [99, 140, 112, 0], 16, 8, 2, 64, 50
    g = torch.Generator().manual_seed(window + tree)
    P, T = 4 * width + 3, sum(new)
    table = torch.randperm(P, generator=g)[:4 * width].reshape(4, width).to(I32)
    parents = [R.random_tree(rng, n) for n in new] if tree else None
    pools = [(torch.randn(P, ps, hkv, D, generator=g) * 64).clamp(-448, 448).to(E4M3) for _ in range(2)]
    exps = [torch.randint(-8, -3, (P, hkv), generator=g).to(torch.int8) for _ in range(2)]
    q = torch.randn(T, hq, D, generator=g).half()
    t = pa.StepTables.empty(4, 4 * width, T, 5 if tree else 0)
    st = status_word()
    pa.pa_v2_build_tables(i32(cached).cuda(), i32(new).cuda(), table.cuda(), ps, t, sliding_window=window, status=st,
                          parents=i32(p for ps_ in parents for p in ps_).cuda() if tree else None)
    got = pa.pa_v2_attention_fp8(q.cuda(), *[x.cuda() for x in pools + exps], t.indices, t.indptr, t.last_page_len,
                                 t.first_page_offset, t.qo_indptr, D ** -0.5, tree_mask=t.tree_mask,
                                 positions=t.positions, sliding_window=window, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and int(t.first_page_offset[0]) > 0
    seen = []
    for r in range(4):
        for i in range(new[r]):
            line = R.ancestors(parents[r], i) if tree else None
            seen.append(F.seen_rows(table[r], ps, 0, cached[r] + new[r], new[r], i, window, 0,
                                    set(line[:window]) if tree else None, len(line) - 1 if tree else i))
    _close(got, F.attention_ref(q, F.values(pools[0], exps[0]), F.values(pools[1], exps[1]), seen, D ** -0.5))


@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_attention_many_rows_nothing_hidden_and_nan_where_it_is_seen(page_size, window, sinks):
    rng = random.Random(5)
    reqs = [(300, 70), (40, 60)]
    c = _attn_case(71, reqs, 8, 2, 128, page_size, torch.bfloat16, window, sinks,
                   trees=[R.random_tree(rng, n, 0.3) for _, n in reqs])
    seen = torch.zeros(c["kp"].shape[0] * page_size, dtype=torch.bool)
    for rows in c["seen"]:
        seen[rows] = True
    for n in ("kp", "vp"):
        c[n].view(torch.uint8).flatten(0, 1)[~seen] = 0x7f
    clean = dict(c, vp=c["vp"].float().nan_to_num(0.0).to(E4M3), kp=c["kp"].float().nan_to_num(0.0).to(E4M3))
    ro, rl, to, tl = ref = _attn_ref(clean)
    st = status_word()
    _close(_run_attn(c, status=st), ref)
    assert int(st) == 0
    hit = [rows[k] for rows in c["seen"][::9] for k in (0, -1)]
    for j, row in enumerate(hit):
        c["vp"].view(torch.uint8).flatten(0, 1)[row, j % 2, (7 * j) % 128] = 0x7f
    out = _run_attn(c)[0].cpu().double()
    flat, nan = c["vp"].float().isnan().flatten(0, 1), torch.zeros(ro.shape, dtype=torch.bool)
    for t, rows in enumerate(c["seen"]):
        nan[t] = flat[rows].any(0).repeat_interleave(4, 0)
    clean["vp"] = c["vp"].float().nan_to_num(0.0).to(E4M3)
    ro, _, to, _ = _attn_ref(clean)
    assert nan.any() and torch.equal(out.isnan(), nan) and ((out - ro).abs() <= to)[~nan].all()


def _long_lists(slots, new, seed=82):
    """One request of 64 KV heads whose list repeats 41 pages; 2048 pages of 16 tokens fit the workspace."""
    c = _attn_case(seed, [(16 * 41 - new, new)], 64, 64, 128, 16, torch.float16)
    ids = c["ids"].repeat(-(-slots // 41))[-slots:]      # (the last ones as they were)
    first = 16 * slots - new
    rows = (ids.long()[:, None] * 16 + torch.arange(16)).flatten().tolist()
    c.update(ids=ids, indptr=i32([0, slots]), seen=[rows[:first + i + 1] for i in range(new)],
             pos=torch.arange(first, first + new, dtype=I32))
    return c


def _some_of(c):
    """The definition's results of some tokens and heads, and what picks them."""
    some, heads = [0, 57, 99], slice(None, None, 31)
    part = dict(c, q=c["q"][some][:, heads], seen=[c["seen"][i] for i in some],
                **{n: c[n][:, :, heads] for n in ("kp", "vp")}, **{n: c[n][:, heads] for n in ("ke", "ve")})
    return _attn_ref(part), lambda got: [x[some][:, heads] for x in got]


@pytest.mark.parametrize("slots,padding", [(1500, 0), (1900, 300), (2048, 1), (2049, 0), (2300, 300)])
def test_attention_many_rows_of_lists_around_the_room(slots, padding):
    """Lists that the host knows to fit, that the device finds to fit, and that do not: the blocks of few rows take
    those, as they do all calls with a workspace without that room."""
    c = _long_lists(slots, 100)
    c["ids"] = torch.cat((c["ids"], torch.zeros(padding, dtype=I32)))
    st = status_word()
    out, lse = _run_attn(c, status=st)
    assert int(st) == 0
    small = _run_attn(c, workspace=pa.attention_fp8_workspace(1, 1, 64, 64, 128))
    if slots > 2048:
        assert torch.equal(out, small[0]) and torch.equal(lse, small[1])
    ref, pick = _some_of(c)
    for got in ((out, lse), small):
        _close(pick(got), ref)


@pytest.mark.parametrize("slots,new", [(1100, 100), (1100, 200)])
def test_attention_overlapping_lists_longer_than_the_room(slots, new):
    """One list for two requests, one without tokens between.  2 * 100 rows on 3 requests are less than 97 each and
    need no room, 2 * 200 are more."""
    c = _long_lists(slots, new)
    ref, pick = _some_of(c)
    c.update(q=torch.cat((c["q"], c["q"])), pos=torch.cat((c["pos"], c["pos"])), indptr=i32([0, slots, 0, slots]),
             lpl=c["lpl"].repeat(3), fpo=c["fpo"].repeat(3), qo=i32([0, new, new, 2 * new]))
    st = status_word()
    out = torch.full((2 * new, 64, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((2 * new, 64), 7.0, device="cuda")
    _run_attn(c, status=st, out=out, lse2_out=lse)
    if new == 100:
        assert int(st) == 0
        for half in (slice(0, new), slice(new, None)):
            _close(pick((out[half], lse[half])), ref)
    else:
        assert int(st) == pa.DEVICE_BAD_TREE and out.eq(0).all() and lse.eq(-math.inf).all()


def test_attention_many_rows_bad_tables_and_graphs():
    def case():
        return _attn_case(91, [(50, 60), (20, 60), (33, 60)], 8, 2, 64, 16, torch.float16)

    ref = _attn_ref(case())
    good = torch.tensor([True] * 60 + [False] * 60 + [True] * 60)
    for page in (-1, 10 ** 6, 2 ** 31 - 1):
        c = case()
        c["ids"][int(c["indptr"][1])] = page
        st = status_word()
        out, lse = _run_attn(c, status=st)
        assert int(st) == pa.DEVICE_BAD_PAGE and out.isfinite().all() and lse.isfinite().all()
        assert ((out.cpu().double() - ref[0]).abs() <= ref[2])[good].all()
    for change in (dict(lpl=0), dict(lpl=17), dict(fpo=-1), dict(fpo=16)):
        c = case()
        for k, v in change.items():
            c[k][1] = v
        st = status_word()
        out, lse = _run_attn(c, status=st)
        assert int(st) == pa.DEVICE_BAD_TREE and out[60:120].eq(0).all() and lse[60:120].eq(-math.inf).all()
        assert ((out.cpu().double() - ref[0]).abs() <= ref[2])[good].all()
    c = case()
    c["indptr"][2] = 10 ** 6
    st = status_word()
    out, lse = _run_attn(c, status=st)
    assert int(st) & pa.DEVICE_BAD_SLOT and out[60:].eq(0).all()
    c = case()
    c["qo"] = i32([0, 60, 50, 180])
    st = status_word()
    _run_attn(c, status=st)
    assert int(st) & pa.DEVICE_BAD_INDPTR
    # rows behind the last token, and a captured call replayed over other lengths
    c = case()
    args = [c[n].cuda() for n in ("q", "kp", "vp", "ke", "ve", "ids", "indptr", "lpl", "fpo", "qo")]
    q = torch.cat((args[0], args[0][:7]))
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 6.0, device="cuda")
    ws = pa.attention_fp8_workspace(187, 3, 8, 2, 64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_v2_attention_fp8(q, *args[1:], c["scale"], out=out, lse2_out=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    _close((out, lse), ref)
    assert out[180:].eq(5.0).all() and lse[180:].eq(6.0).all()
    d = _attn_case(92, [(70, 10), (10, 150), (3, 20)], 8, 2, 64, 16, torch.float16)
    n = d["kp"].shape[0]
    assert n <= args[1].shape[0] and len(d["ids"]) <= len(args[5])
    for x, k in zip(args[1:5], ("kp", "vp", "ke", "ve")):
        x[:n] = d[k].cuda()
    q[:180] = d["q"].cuda()
    args[5][:len(d["ids"])] = d["ids"].cuda()
    for x, k in zip(args[6:], ("indptr", "lpl", "fpo", "qo")):
        x.copy_(d[k])
    graph.replay()
    torch.cuda.synchronize()
    _close((out, lse), _attn_ref(d))


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30, 3.0])
def test_attention_other_scales(scale):
    c = _attn_case(21, [(300, 2), (31, 1)], 8, 2, 128, 16, torch.float16)
    c["scale"] = scale
    if scale == 3.0:            # (sharp scores: the reference's own tolerance grows with them)
        c["q"] = c["q"] * 4
    if scale < 0:
        c2 = dict(c, q=-c["q"], scale=-scale)
        _close(_run_attn(c), _attn_ref(c2))
    else:
        _check_attn(c)


def test_attention_small_weights_still_count():
    """One key far above the others, whose weights of 2^-20 each make up a part of the sum that an f16 without a shift
    would lose."""
    c = _attn_case(22, [(4095, 1)], 1, 1, 64, 16, torch.float16)
    kp = torch.zeros(c["kp"].shape)
    kp[int(c["ids"][3]), 5, 0, 0] = 256.0
    c["kp"], c["ke"] = kp.to(E4M3), torch.full_like(c["ke"], -4)
    c["vp"] = torch.full_like(c["vp"].float(), 64.0).to(E4M3)
    c["vp"][int(c["ids"][3]), 5] = torch.zeros(1, 64).to(E4M3)
    c["ve"] = torch.full_like(c["ve"], -6)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][0, 0, 0] = 20 * math.log(2.0) / 16.0
    c["scale"] = 1.0
    out, _ = _check_attn(c)
    assert 0.003 < float(out[0, 0, 0]) < 0.005


@pytest.mark.parametrize("weight", [24, 28, 31, 34])
def test_attention_weights_below_the_normal_halves(weight):
    """One key at each request's begin far above 2047 others of weight 2^-24 .. 2^-34 each, all of the result since its own
    value is zero.  P is a half 2^11 at the row's offset: below 2^-25 of it a subnormal one, off by half a step of 2^-24,
    2^-36 of the offset.  16 requests of 64 heads over the same pages: runs of more than 30 tiles a warp."""
    B, H, D, N = 16, 64, 64, 2047
    c = _attn_case(25, [(N, 1)], H, H, D, 16, torch.float16)
    kp = torch.zeros(c["kp"].shape)
    kp[int(c["ids"][0]), 3, :, 0] = 256.0
    vp = torch.full_like(kp, 448.0)
    vp[int(c["ids"][0]), 3] = 0.0
    c.update(kp=kp.to(E4M3), vp=vp.to(E4M3), ke=torch.full_like(c["ke"], -4), ve=torch.full_like(c["ve"], 7), scale=1.0)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][..., 0] = weight * math.log(2.0) / 16.0
    one = {n: c[n][:, :, :1] for n in ("kp", "vp")} | {n: c[n][:, :1] for n in ("ke", "ve")}
    ro, rl, to, tl = _attn_ref(dict(c, q=c["q"][:, :1], **one))
    to = to + N * 2.0 ** -36 * 57344.0
    assert (to < ro.abs() / 2).all()
    many = dict(c, q=c["q"].repeat(B, 1, 1), ids=c["ids"].repeat(B), indptr=i32(128 * r for r in range(B + 1)),
                lpl=c["lpl"].repeat(B), fpo=c["fpo"].repeat(B), qo=i32(range(B + 1)), pos=c["pos"].repeat(B))
    out, lse = (x.cpu().double() for x in _run_attn(many))
    assert ((out - ro).abs() <= to).all(), (float((out - ro).abs().max()), float(to.max()))
    assert ((lse - rl).abs() <= tl).all()


@pytest.mark.parametrize("dtype,size,scale", [(torch.float16, 1.0, 1e38), (torch.float16, 30000.0, 1e38),
                                              (torch.float16, 65504.0, -2e38), (torch.bfloat16, 60000.0, 2.3e38),
                                              (torch.bfloat16, 2.0 ** 100, 1e38)])
@pytest.mark.parametrize("n", [1, 3, 60])
def test_attention_scores_of_zero_at_the_largest_scales(dtype, size, scale, n):
    """A scale that f32 and its logarithm's base hold, rows of q however large, keys of zero: every score is zero."""
    c = _attn_case(26, [(100, n), (3, n)], 8, 2, 128, 16, dtype)
    c["q"] = torch.full_like(c["q"], size)
    c["q"][:, :, ::2] = -1.0
    c["kp"], c["scale"] = torch.zeros(c["kp"].shape).to(E4M3), scale
    _close(_run_attn(c), _attn_ref(dict(c, scale=1.0)))


@pytest.mark.parametrize("dtype", DT)
def test_attention_ends_of_the_ranges(dtype):
    """Exponents from end to end, out of range ones, codes from the smallest to the largest, large and tiny rows of q."""
    c = _attn_case(23, [(130, 2), (64, 1)], 4, 2, 128, 16, dtype)
    g = torch.Generator().manual_seed(5)
    for n in ("kp", "vp"):
        x = torch.randint(0, 256, c[n].shape, generator=g, dtype=torch.uint8)
        c[n] = torch.where((x & 0x7f) == 0x7f, x ^ 1, x).view(E4M3)
    c["ve"] = torch.randint(-15, 8, c["ve"].shape, generator=g).to(torch.int8)
    c["ke"] = torch.randint(-15, -9, c["ke"].shape, generator=g).to(torch.int8)
    c["ve"][0, 0], c["ve"][1, 1], c["ke"][2, 0] = 127, -128, -100
    c["q"][0] *= 2.0 ** -20
    c["q"][1] *= 2.0 ** 5
    _check_attn(c)


def test_attention_bad_tables_are_contained_and_reported():
    def case():
        return _attn_case(31, [(50, 1), (20, 2), (33, 1)], 4, 2, 64, 16, torch.float16)

    c = case()
    ref = _attn_ref(c)
    others = [0, 3]                         # tokens of the requests that stay good

    def run(c, want, zero=(1, 2), **kw):
        st = status_word()
        out, lse = _run_attn(c, status=st, **kw)
        assert int(st) == want, (int(st), want)
        for t in others:
            assert ((out[t].cpu().double() - ref[0][t]).abs() <= ref[2][t]).all()
        if zero:
            assert (out[list(zero)] == 0).all() and (lse[list(zero)] == -math.inf).all()
        return out, lse

    for page in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        c = case()
        c["ids"][int(c["indptr"][1])] = page
        out, lse = run(c, pa.DEVICE_BAD_PAGE, zero=())
        assert out.isfinite().all() and lse.isfinite().all()
    for lpl in (0, -3, 17, 2 ** 31 - 1):
        c = case()
        c["lpl"][1] = lpl
        run(c, pa.DEVICE_BAD_TREE)
    for fpo in (-1, 16, 2 ** 31 - 1):
        c = case()
        c["fpo"][1] = fpo
        run(c, pa.DEVICE_BAD_TREE)
    c = case()                              # more new tokens than listed ones
    c["indptr"] = i32([0, 4, 4, 7])
    c["ids"] = torch.cat((c["ids"][:4], c["ids"][6:]))
    run(c, pa.DEVICE_BAD_TREE)
    c = case()                              # slots past the list
    c["indptr"][1:3] = i32([4, 10 ** 6])
    st = status_word()
    _run_attn(c, status=st)
    assert int(st) & pa.DEVICE_BAD_SLOT
    c = case()                              # new tokens past the call's
    c["qo"] = i32([0, 1, 3, 100])
    st = status_word()
    _run_attn(c, status=st)
    assert int(st) == pa.DEVICE_BAD_INDPTR
    c = case()
    c["qo"] = i32([0, 3, 1, 4])
    st = status_word()
    _run_attn(c, status=st)
    assert int(st) & pa.DEVICE_BAD_INDPTR
    c = case()                              # sinks of a table that does not begin at the request's start
    c["window"], c["sinks"] = 4096, 4
    c["fpo"][1], c["lpl"][1] = 1, c["lpl"][1] + 1
    run(c, pa.DEVICE_BAD_TREE)
    c = case()
    c["window"], c["sinks"] = 4096, 4
    c["pos"][1] += 1
    run(c, pa.DEVICE_BAD_TREE)
    c = case()                              # a window that the table does not hold
    c["window"] = 40
    c["pos"][1:3] += 100
    ref = _attn_ref(dict(case(), seen=[rows[-40:] for rows in case()["seen"]]))
    run(c, pa.DEVICE_BAD_TREE)


def test_attention_tables_that_claim_pages_and_tokens_again_stay_in_bounds():
    c = _attn_case(32, [(400, 3)], 4, 2, 64, 16, torch.float16)
    B, n = 40, len(c["ids"])
    c["indptr"] = i32([0, n] * 20 + [0])
    c["lpl"], c["fpo"] = i32([16] * B), i32([0] * B)
    c["qo"] = i32([0, 3] * 20 + [0])
    st = status_word()
    out, lse = _run_attn(c, status=st)
    assert int(st) & (pa.DEVICE_BAD_INDPTR | pa.DEVICE_BAD_SLOT)


def test_attention_more_new_tokens_than_mask_bits():
    c = _attn_case(33, [(10, 40)], 4, 2, 64, 16, torch.float16, trees=[R.random_tree(random.Random(1), 40)])
    c["mask"] = c["mask"][:, :1].contiguous()
    st = status_word()
    out, lse = _run_attn(c, status=st)
    assert int(st) == pa.DEVICE_BAD_TREE and (out == 0).all() and (lse == -math.inf).all()


def test_attention_without_positions():
    c = _attn_case(34, [(300, 3), (20, 1)], 4, 2, 64, 16, torch.float16, 50, 4)
    args = [c[n].cuda() for n in ("q", "kp", "vp", "ke", "ve", "ids", "indptr", "lpl", "fpo", "qo")]
    got = pa.pa_v2_attention_fp8(*args, c["scale"], sliding_window=50, sinks=4)
    _close(got, _attn_ref(c))
    with pytest.raises(ValueError, match="positions"):
        pa.pa_v2_attention_fp8(*args, c["scale"], sliding_window=50, tree_mask=torch.zeros(4, 1, dtype=I32).cuda())


def test_attention_repeats_itself_and_takes_any_workspace():
    c = _attn_case(35, [(9000, 2), (700, 1), (3, 1)], 8, 2, 128, 16, torch.bfloat16)
    a = _run_attn(c)
    n = pa.pa_v2_attention_fp8_workspace(4, 3, 8, 2, 128)
    for fill in (0, 255):
        b = _run_attn(c, workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    with pytest.raises(pa.PaError) as e:
        _run_attn(c, workspace=torch.zeros(n - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pa.PA_ECAPACITY


def test_attention_workspace_for_other_sizes():
    """A workspace made for the most tokens and requests serves every smaller call, also one whose tokens all belong to
    one request (which would like a larger one)."""
    ws = pa.attention_fp8_workspace(128, 128, 8, 2, 128)
    for reqs in ([(300, 128)], [(300, 100), (7, 28)], [(20, 1)] * 128):
        _check_attn(_attn_case(36, reqs, 8, 2, 128, 16, torch.bfloat16), workspace=ws)
    large = pa.attention_fp8_workspace(256, 2, 8, 2, 128)
    assert large.numel() > ws.numel()
    for reqs in ([(300, 128), (7, 128)], [(300, 128)], [(20, 1)] * 2):
        _check_attn(_attn_case(37, reqs, 8, 2, 128, 16, torch.bfloat16), workspace=large)


def test_attention_without_a_new_token():
    c = _attn_case(38, [(30, 0), (0, 0), (5, 0)], 4, 2, 64, 16, torch.float16)
    out, lse = torch.full((5, 4, 64), 5.0, dtype=torch.float16, device="cuda"), torch.full((5, 4), 6.0, device="cuda")
    st = status_word()
    _run_attn(c, pad=5, out=out, lse2_out=lse, status=st)
    assert int(st) == 0 and out.eq(5.0).all() and lse.eq(6.0).all()


@pytest.mark.parametrize("hkv", [67, 96, 130])
@pytest.mark.parametrize("ctx", [40, 700])
def test_attention_many_kv_heads(hkv, ctx):
    _check_attn(_attn_case(hkv, [(ctx, 1), (3, 2), (2 * ctx, 1)], hkv, hkv, 64, 16, torch.float16))


def test_attention_two_calls_at_once_and_two_graphs_side_by_side():
    cases = [_attn_case(40 + k, [(3000, 2), (50 + k, 1)], 8, 2, 128, 16, DT[k]) for k in range(2)]
    alone = [[x.clone() for x in _run_attn(c)] for c in cases]
    streams, graphs, outs, keep = [torch.cuda.Stream() for _ in cases], [], [], []
    for c, s in zip(cases, streams):
        args = [c[n].cuda() for n in ("q", "kp", "vp", "ke", "ve", "ids", "indptr", "lpl", "fpo", "qo")]
        out, lse = torch.zeros_like(args[0]), torch.zeros(args[0].shape[:2], device="cuda")
        ws = pa.attention_fp8_workspace(args[0].shape[0], 2, 8, 2, 128)
        keep.append((args, ws))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pa.pa_v2_attention_fp8(*args, c["scale"], out=out, lse2_out=lse, workspace=ws)
        graphs.append(graph)
        outs.append((out, lse))
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for want, got in zip(alone, outs):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(want, got))
    for o, l in outs:
        o.zero_(), l.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, (args, ws), (out, lse) in zip(cases, streams, keep, outs):
            pa.pa_v2_attention_fp8(*args, c["scale"], out=out, lse2_out=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for want, got in zip(alone, outs):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(want, got))


@pytest.mark.parametrize("page_size", [16, 5])
def test_pools_of_more_elements_than_32_bits_count(page_size):
    D, hkv = 128, 8
    P = (2 ** 32 + 2 ** 22) // (page_size * hkv * D)
    c = _attn_case(50, [(90, 2), (33, 1)], 8, hkv, D, page_size, torch.float16)
    n = c["kp"].shape[0]
    ids = c["ids"].clone()
    big = dict(c, ids=ids + (P - n))
    pools = []
    for name in ("kp", "vp"):
        x = torch.zeros(P, page_size, hkv, D, dtype=torch.uint8, device="cuda")
        x[P - n:] = c[name].view(torch.uint8).cuda()
        pools.append(x.view(E4M3))
    for name in ("ke", "ve"):
        e = torch.zeros(P, hkv, dtype=torch.int8, device="cuda")
        e[P - n:] = c[name].cuda()
        pools.append(e)
    st = status_word()
    got = pa.pa_v2_attention_fp8(c["q"].cuda(), *pools, big["ids"].cuda(), c["indptr"].cuda(), c["lpl"].cuda(),
                                 c["fpo"].cuda(), c["qo"].cuda(), c["scale"], status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    _close(got, _attn_ref(c))
    # an append behind them
    a = _append_case(51, [(0, 3)], page_size, 8, hkv, D, 128, torch.bfloat16, True)
    small = [a[k].cuda() for k in ("kp", "vp", "ke", "ve")]
    _run_append(a, cache=small)
    m = a["kp"].shape[0]
    for x, y in zip(pools, ("kp", "vp", "ke", "ve")):
        x[P - m:].view(torch.uint8).copy_(a[y].view(torch.uint8))
    _run_append(dict(a, slots=a["slots"] + (P - m) * page_size), cache=pools)
    for x, y in zip(small, pools):
        assert torch.equal(x.view(torch.uint8), y[P - m:].view(torch.uint8))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("window", [5, 40, 300])
def test_sliding_tables_feed_the_attention(window, tree):
    """pa_v2_build_tables_sliding's trimmed tables, cut masks and positions, as the 16-bit attention takes them."""
    rng = random.Random(window)
    cached, new, ps, hq, hkv, D = [700, 33, 0, 90], [9, 40, 12, 0], 16, 4, 2, 64
    g = torch.Generator().manual_seed(window)
    width = 48
    table = torch.randperm(4 * width + 3, generator=g)[:4 * width].reshape(4, width).to(I32)
    parents = [R.random_tree(rng, n) for n in new] if tree else None
    P, T = 4 * width + 3, sum(new)
    pools, exps = [], []
    for _ in range(2):
        pools.append((torch.randn(P, ps, hkv, D, generator=g) * 64).clamp(-448, 448).to(E4M3))
        exps.append(torch.randint(-8, -3, (P, hkv), generator=g).to(torch.int8))
    q = torch.randn(T, hq, D, generator=g).bfloat16()
    t = pa.StepTables.empty(4, 4 * width, T, 2 if tree else 0)
    st = status_word()
    pa.pa_v2_build_tables(i32(cached).cuda(), i32(new).cuda(), table.cuda(), ps, t, sliding_window=window, status=st,
                          parents=i32(p for ps_ in parents for p in ps_).cuda() if tree else None)
    got = pa.pa_v2_attention_fp8(q.cuda(), *[x.cuda() for x in pools + exps], t.indices, t.indptr, t.last_page_len,
                                 t.first_page_offset, t.qo_indptr, D ** -0.5, tree_mask=t.tree_mask,
                                 positions=t.positions, sliding_window=window, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    seen = []
    for r in range(4):
        for i in range(new[r]):
            line = R.ancestors(parents[r], i)[:window] if tree else None
            depth = len(R.ancestors(parents[r], i)) - 1 if tree else i
            seen.append(F.seen_rows(table[r], ps, 0, cached[r] + new[r], new[r], i, window, 0,
                                    set(line) if tree else None, depth))
    _close(got, F.attention_ref(q, F.values(pools[0], exps[0]), F.values(pools[1], exps[1]), seen, D ** -0.5))


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 4)])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_from_lengths_to_outputs(graph, window, sinks):
    """Tables, append and attention over several steps of several requests, in a graph or not: a prompt's chunk, then
    single tokens.  Each step's outputs are those of the definition over the cache as it stands."""
    B, hq, hkv, D, ps, steps = 3, 8, 2, 64, 16, 6
    g = torch.Generator().manual_seed(17)
    width = 6
    table = torch.randperm(40, generator=g)[:B * width].reshape(B, width).to(I32)
    cache = [torch.zeros(40, ps, hkv, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.zeros(40, hkv, dtype=torch.int8, device="cuda") for _ in range(2)]
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float32) / (D // 2)))
    cap = 60
    t = pa.StepTables.empty(B, B * width, cap, 0)
    x = torch.zeros(cap, hq + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
    cached, new = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    q2, out = torch.zeros(cap, hq, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(cap, hq, D, dtype=torch.bfloat16, device="cuda")
    lse, st, dtab = torch.zeros(cap, hq, device="cuda"), status_word(), table.cuda()
    ws, dfreq = pa.attention_fp8_workspace(cap, B, hq, hkv, D), freq.cuda()

    def step():
        pa.pa_v2_build_tables(cached, new, dtab, ps, t, status=st)
        pa.pa_v2_qk_rope_append_fp8(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], t.positions, t.slots, dfreq, *cache,
                                    q_out=q2, status=st)
        pa.pa_v2_attention_fp8(q2, *cache, t.indices, t.indptr, t.last_page_len, t.first_page_offset, t.qo_indptr,
                               D ** -0.5, positions=t.positions, sliding_window=window, sinks=sinks, out=out,
                               lse2_out=lse, workspace=ws, status=st)

    captured = None
    if graph:
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    lens = [0, 0, 0]
    for s in range(steps):
        news = [30, 11, 17] if s == 0 else [1, 1, 2 if s == 2 else 1]
        cached.copy_(i32(lens))
        new.copy_(i32(news))
        x.copy_((torch.randn(cap, hq + 2 * hkv, D, generator=g) * (1 + s)).bfloat16())
        before = [c.cpu().clone() for c in cache]
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        assert int(st) == 0
        T = sum(news)
        slots, pos = t.slots.cpu(), t.positions.cpu()
        case = dict(q=x[:, :hq].cpu(), k=x[:, hq:hq + hkv].cpu(), v=x[:, hq + hkv:].cpu(), qw=None, kw=None, eps=0.0,
                    pos=pos, slots=slots, kp=before[0], vp=before[1], ke=before[2], ve=before[3], freq=freq)
        _check_append(case, q2, cache)
        seen = []
        for r in range(B):
            for i in range(news[r]):
                seen.append(F.seen_rows(table[r], ps, 0, lens[r] + news[r], news[r], i, window, sinks))
        ref = F.attention_ref(q2[:T].cpu(), F.values(cache[0].cpu(), cache[2].cpu()),
                              F.values(cache[1].cpu(), cache[3].cpu()), seen, D ** -0.5)
        _close((out, lse), ref)
        lens = [a + b for a, b in zip(lens, news)]
