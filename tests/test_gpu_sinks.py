"""GPU: attention of new tokens under a sliding window with sinks over 16-bit pools (pa_v2_tree_attention_sinks) against
plain 64-bit references, each token over the rows that it sees."""
import math
import random

import pytest
import torch

import fp8_reference as F
import step_reference as R
from paged_attention_decode_gb300 import pa_v2 as pa

pytestmark = pytest.mark.gpu

I32 = torch.int32
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


def _case(seed, reqs, window, sinks, hq, hkv, D, page_size, dtype, trees=None, give_back=True):
    """reqs: (cached, new) per request, the whole of each listed; pages that nobody sees given back."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-(c + n) // page_size) for c, n in reqs]
    P = sum(counts) + 3
    ids = torch.randperm(P, generator=g)[:sum(counts)].to(I32)
    kp, vp = (torch.randn(P, page_size, hkv, D, generator=g).to(dtype) for _ in range(2))
    indptr = prefix(counts)
    seen, positions, rows = [], [], []
    words = max(1, -(-max(n for _, n in reqs) // 32))
    for r, (c, n) in enumerate(reqs):
        for i in range(n):
            line = R.ancestors(trees[r], i) if trees else None
            depth = len(line) - 1 if trees else i
            if trees:
                line = line[:window]
                rows.append(R.words_of(sum(1 << j for j in line), words))
            seen.append(F.seen_rows(ids[indptr[r]:indptr[r + 1]], page_size, 0, c + n, n, i, window, sinks,
                                    set(line) if trees else None, depth))
            positions.append(c + depth)
    if give_back:
        used = {row // page_size for s in seen for row in s}
        for s in range(len(ids)):
            if int(ids[s]) not in used:
                ids[s] = -1
    T = sum(n for _, n in reqs)
    return dict(q=(1.4 * torch.randn(T, hq, D, generator=g)).to(dtype), kp=kp, vp=vp, ids=ids, indptr=i32(indptr),
                lpl=i32((c + n - 1) % page_size + 1 if c + n else 0 for c, n in reqs), fpo=i32([0] * len(reqs)),
                qo=i32(prefix(n for _, n in reqs)), mask=torch.tensor(rows, dtype=I32).reshape(T, words) if trees else None,
                pos=i32(positions), window=window, sinks=sinks, scale=D ** -0.5, seen=seen)


def _run(c, **kw):
    out, lse = pa.pa_v2_tree_attention(
        c["q"].cuda(), c["kp"].cuda(), c["vp"].cuda(), c["ids"].cuda(), c["indptr"].cuda(), c["lpl"].cuda(),
        c["fpo"].cuda(), c["qo"].cuda(), c["scale"], tree_mask=None if c["mask"] is None else c["mask"].cuda(),
        positions=c["pos"].cuda(), sliding_window=c["window"], sinks=c["sinks"], **kw)
    torch.cuda.synchronize()
    return out, lse


def _ref(c):
    return F.attention_ref(c["q"], c["kp"], c["vp"], c["seen"], c["scale"])


def _check(c, ref=None):
    st = status_word()
    out, lse = (x.cpu().double() for x in _run(c, status=st))
    assert int(st) == 0
    ro, rl, to, tl = ref or _ref(c)
    fine = rl > -math.inf
    assert torch.equal(lse > -math.inf, fine)
    assert ((out - ro).abs() <= to).all(), float(((out - ro).abs() - to).max())
    assert ((lse - rl).abs() <= tl)[fine].all(), float((lse - rl)[fine].abs().max())
    return out, lse


CASES = [
    ([(3000, 1)], 64, 4), ([(3000, 1)], 1, 1), ([(3000, 5)], 300, 200), ([(700, 1), (130, 1), (5, 1), (0, 1), (300, 0)], 128, 4),
    ([(900, 40), (127, 3), (0, 12)], 130, 128), ([(2000, 7)], 256, 129), ([(500, 3)], 100000, 7), ([(2000, 2)], 5, 1900),
    ([(300, 300)], 40, 3), ([(1000, 260)], 500, 256), ([(128, 1), (129, 1), (255, 1), (256, 1), (257, 2)], 128, 1),
    ([(20, 50)], 4, 33), ([(600, 2)] * 40, 200, 16),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("reqs,window,sinks", CASES)
@pytest.mark.parametrize("page_size,D,hq,hkv", [(16, 128, 8, 2), (5, 64, 6, 2)])
def test_chains(reqs, window, sinks, page_size, D, hq, hkv, dtype):
    _check(_case(len(reqs) + window + sinks, reqs, window, sinks, hq, hkv, D, page_size, dtype))


@pytest.mark.parametrize("page_size", [1, 3, 8, 48, 64, 256])
def test_page_sizes(page_size):
    _check(_case(page_size, [(1500, 4), (90, 1), (300, 9)], 140, 10, 4, 2, 128, page_size, torch.float16))


@pytest.mark.parametrize("window,sinks", [(20, 4), (70, 150), (3, 1)])
@pytest.mark.parametrize("page_size", [16, 5])
def test_trees(window, sinks, page_size):
    rng = random.Random(window)
    reqs = [(700, 60), (100, 33), (0, 40), (260, 1)]
    trees = [R.random_tree(rng, n) for _, n in reqs]
    trees[1] = [i - 1 if i % 9 else max(i - 4, -1) for i in range(33)]     # deeper than the window
    _check(_case(3, reqs, window, sinks, 8, 2, 128, page_size, torch.bfloat16, trees))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("tree", [False, True])
def test_nothing_hidden_reaches_a_result(bad, page_size, tree):
    rng = random.Random(2)
    reqs = [(700, 20), (300, 7), (60, 12)]
    trees = [R.random_tree(rng, n) for _, n in reqs] if tree else None
    c = _case(4, reqs, 150, 9, 8, 2, 64, page_size, torch.bfloat16, trees, give_back=False)
    ref = _ref(c)
    seen = torch.zeros(c["kp"].shape[0] * page_size, dtype=torch.bool)
    for rows in c["seen"]:
        seen[rows] = True
    for n in ("kp", "vp"):
        c[n].flatten(0, 1)[~seen] = bad
    _check(c, ref)


@pytest.mark.parametrize("page_size", [16, 5])
@pytest.mark.parametrize("n", [1, 30])
def test_infinite_values_reach_the_rows_that_see_them_and_no_other(page_size, n):
    reqs = [(700, n), (200, n)]
    c = _case(5, reqs, 100, 6, 4, 2, 128, page_size, torch.float16)
    # a sink, a row that only some of the window's tokens see, a new token
    hit = [c["seen"][0][2], c["seen"][0][6], c["seen"][n - 1][-1], c["seen"][-1][3]]
    for j, row in enumerate(hit):
        c["vp"].flatten(0, 1)[row, j % 2, 5 * j] = -math.inf if j % 2 else math.inf
    st = status_word()
    out, lse = (x.cpu().double() for x in _run(c, status=st))
    assert int(st) == 0
    clean = dict(c, vp=torch.where(c["vp"].isfinite(), c["vp"], 0.0))
    ro, rl, to, tl = _ref(clean)
    want = torch.zeros_like(ro)
    flat = torch.where(c["vp"].isfinite(), 0.0, c["vp"]).flatten(0, 1).double()
    for t, rows in enumerate(c["seen"]):
        want[t] = flat[rows].sum(0).repeat_interleave(2, 0)
    inf = want.isinf()
    assert inf.any() and torch.equal(out[inf], want[inf])
    assert ((out - ro).abs() <= to)[~inf].all() and ((lse - rl).abs() <= tl).all()


def test_refused_tables():
    def run(change, want=pa.DEVICE_BAD_TREE):
        c = _case(6, [(50, 1), (20, 2), (33, 1)], 24, 4, 4, 2, 64, 16, torch.float16)
        ref = _ref(c)
        change(c)
        st = status_word()
        out, lse = (x.cpu().double() for x in _run(c, status=st))
        assert int(st) == want
        for t in (0, 3):
            assert ((out[t] - ref[0][t]).abs() <= ref[2][t]).all()
        assert out[1:3].eq(0).all() and lse[1:3].eq(-math.inf).all()

    def trimmed(c):
        c["fpo"][1] = 1

    def moved(c):
        c["pos"][1] += 1

    def behind(c):
        c["pos"][1] -= 1

    for change in (trimmed, moved, behind):
        run(change)
    with pytest.raises(ValueError, match="sinks"):
        c = _case(6, [(50, 1)], 24, 4, 4, 2, 64, 16, torch.float16)
        c["window"] = 0
        _run(c)


def test_sinks_that_never_bind_equal_the_other_calls():
    """More sinks than tokens, or a window over all of them: what the call without a window gives."""
    c = _case(7, [(900, 5), (3, 2)], 10, 2000, 8, 2, 128, 16, torch.bfloat16)
    a = _run(c)
    b = pa.pa_v2_tree_attention(c["q"].cuda(), c["kp"].cuda(), c["vp"].cuda(), c["ids"].cuda(), c["indptr"].cuda(),
                                c["lpl"].cuda(), c["fpo"].cuda(), c["qo"].cuda(), c["scale"])
    _check(c)
    assert (a[0].double() - b[0].double()).abs().max() < 0.02 and (a[1] - b[1]).abs().max() < 1e-3


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_single_tokens_with_pages_given_back(graph):
    """Tables of whole requests whose middle pages the program has taken back, append and attention, step by step."""
    B, hq, hkv, D, ps, window, sinks = 3, 8, 2, 64, 4, 9, 5
    g = torch.Generator().manual_seed(1)
    lens, width = [40, 7, 0], 16
    table = torch.randperm(60, generator=g)[:B * width].reshape(B, width).to(I32)
    kp, vp = (torch.randn(60, ps, hkv, D, generator=g).half().cuda() for _ in range(2))
    dtab, t, st = table.clone().cuda(), pa.StepTables.empty(B, B * width, B), status_word()
    x = torch.zeros(B, hq + 2 * hkv, D, dtype=torch.float16, device="cuda")
    cached, new = i32(lens).cuda(), i32([1] * B).cuda()
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float32) / (D // 2))).cuda()
    q2, out, lse = torch.zeros(B, hq, D).half().cuda(), torch.zeros(B, hq, D).half().cuda(), torch.zeros(B, hq).cuda()
    ws = pa.tree_attention_workspace(B, B, hq, hkv, D)

    def step():
        pa.pa_v2_build_tables(cached, new, dtab, ps, t, status=st)
        pa.pa_v2_qk_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], t.positions, t.slots, freq, kp, vp,
                                q_out=q2, status=st)
        pa.pa_v2_tree_attention(q2, kp, vp, t.indices, t.indptr, t.last_page_len, t.first_page_offset, t.qo_indptr,
                                D ** -0.5, positions=t.positions, sliding_window=window, sinks=sinks, out=out,
                                lse2_out=lse, workspace=ws, status=st)

    captured = None
    if graph:
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for _ in range(12):
        gone = dtab.cpu()
        for r in range(B):
            for p in range(-(-lens[r] // ps)):
                if p * ps >= sinks and (p + 1) * ps <= lens[r] - window + 1:
                    gone[r, p] = -1
        dtab.copy_(gone)
        cached.copy_(i32(lens))
        x.copy_(torch.randn(B, hq + 2 * hkv, D, generator=g).half())
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        assert int(st) == 0
        seen = [F.seen_rows(table[r], ps, 0, lens[r] + 1, 1, 0, window, sinks) for r in range(B)]
        ro, rl, to, tl = F.attention_ref(q2.cpu(), kp.cpu(), vp.cpu(), seen, D ** -0.5)
        assert ((out.cpu().double() - ro).abs() <= to).all() and ((lse.cpu().double() - rl).abs() <= tl).all()
        lens = [n + 1 for n in lens]
