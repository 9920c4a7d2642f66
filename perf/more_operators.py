"""Measured cases of the 8-bit cache (append and attention) and of attention with a sliding window and sinks.

Each case is one pass through one operator of a serving step over a paged KV cache:

- ``append8``: per-head norm of q and k, position rotation, and the append of k and v to pools of e4m3 codes with one
  power-of-two exponent for each page and KV head (a value is code * 2^exponent);
- ``attn8``: attention of each request's new tokens over such pools, whole or with a window and sinks;
- ``sink16``: attention of the new tokens over 16-bit pools where each sees the first tokens (the sinks) and a sliding
  window up to itself.

``run`` computes the operator in elementary torch operations, or, with ``own`` set, makes the calls a user
makes of ``paged_attention_decode_gb300.pa_v2``.  A case's sizes are fixed by the case (its ``lens`` number
seeds the ragged lengths and the shapes of the trees); the seed of ``prepare`` decides the values, the
physical pages and the order of the requests.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"f16": 2, "bf16": 2, "f32": 4}
CODE = torch.float8_e4m3fn
CODE_MAX = 448.0                 # largest e4m3 value
EXP_LO, EXP_HI = -15, 7          # exponents of a page: every code * 2^exponent is a binary16 number
DEVICE = "cuda"


def listed():
    return [
        # single-token decode of a small batch, pages partly filled: rotation only, latency counts
        dict(name="append8_decode_b8", op="append8", batch=8, ctx_lo=100, ctx_hi=32768, new_lo=1, new_hi=1, hq=32,
             hkv=8, dim=128, rot=128, interleaved=False, norm=False, dtype="f16", page_size=16, pad=0, lens=1),
        # 32 requests with 64 drafted tokens each to verify, normed heads
        dict(name="append8_verify_2048", op="append8", batch=32, ctx_lo=512, ctx_hi=131072, new_lo=64, new_hi=64,
             hq=32, hkv=8, dim=128, rot=128, interleaved=False, norm=True, dtype="bf16", page_size=16, pad=0, lens=2),
        # chunks of two prompts
        dict(name="append8_prompt_16384", op="append8", batch=2, ctx_lo=1, ctx_hi=65536, new_lo=8192, new_hi=8192,
             hq=32, hkv=8, dim=128, rot=128, interleaved=False, norm=True, dtype="bf16", page_size=16, pad=0, lens=3),
        # f32 activations, a partial, interleaved rotation, few heads, an odd page size, padded tokens behind the last
        dict(name="append8_odd_f32", op="append8", batch=19, ctx_lo=1, ctx_hi=1000000, new_lo=1, new_hi=79, hq=12,
             hkv=4, dim=64, rot=32, interleaved=True, norm=True, dtype="f32", page_size=5, pad=37, lens=4),
        # the smallest attention call: one token of one request over a short context, latency bound
        dict(name="attn8_b1_1k", op="attn8", batch=1, ctx_lo=1024, ctx_hi=1024, new_lo=1, new_hi=1, chain=True, hq=32,
             hkv=8, dim=128, page_size=16, window=0, sinks=0, dtype="f16", lens=5),
        # the 32K single-token decode shape
        dict(name="attn8_b1_32k", op="attn8", batch=1, ctx_lo=32768, ctx_hi=32768, new_lo=1, new_hi=1, chain=True,
             hq=32, hkv=8, dim=128, page_size=16, window=0, sinks=0, dtype="f16", lens=6),
        # a serving batch of single tokens over ragged contexts: the most bytes
        dict(name="attn8_b64_ragged", op="attn8", batch=64, ctx_lo=1024, ctx_hi=32768, new_lo=1, new_hi=1, chain=True,
             hq=32, hkv=8, dim=128, page_size=16, window=0, sinks=0, dtype="bf16", lens=7),
        # chains of five drafted tokens under a window with sinks, pages between the two given back
        dict(name="attn8_b32_chain5_sinks", op="attn8", batch=32, ctx_lo=512, ctx_hi=65536, new_lo=5, new_hi=5,
             chain=True, hq=32, hkv=8, dim=128, page_size=16, window=4096, sinks=4, dtype="bf16", lens=8),
        # chunks of four prompts over what is cached of them: the most products
        dict(name="attn8_b4_256tok_8k", op="attn8", batch=4, ctx_lo=8192, ctx_hi=8192, new_lo=256, new_hi=256,
             chain=True, hq=32, hkv=8, dim=128, page_size=16, window=0, sinks=0, dtype="bf16", lens=9),
        # odd everything: page size 5, three query heads per KV head, head_dim 64, trees over short ragged contexts
        dict(name="attn8_b7_odd", op="attn8", batch=7, ctx_lo=33, ctx_hi=2999, new_lo=1, new_hi=33, chain=False, hq=24,
             hkv=8, dim=64, page_size=5, window=0, sinks=0, dtype="f16", lens=10),
        # single tokens of 64 long requests under a window with sinks over a bf16 cache
        dict(name="sink16_b64_decode", op="sink16", batch=64, ctx_lo=512, ctx_hi=65536, new_lo=1, new_hi=1, chain=True,
             hq=32, hkv=8, dim=128, page_size=16, window=4096, sinks=4, dtype="bf16", lens=11),
        # drafted trees under a short window with a few more sinks, an f16 cache of large pages
        dict(name="sink16_b16_tree", op="sink16", batch=16, ctx_lo=100, ctx_hi=16384, new_lo=1, new_hi=64, chain=False,
             hq=32, hkv=8, dim=128, page_size=64, window=1024, sinks=64, dtype="f16", lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append8", "attn8", "attn8", "sink16"])
    hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 3, 4, 4, 7, 8])
    if hkv * group > 40:
        group = 4
    dim = rng.choice([64, 128, 128])
    page = rng.choice([1, 5, 8, 16, 16, 16, 48, 64])
    sizes = dict(hq=hkv * group, hkv=hkv, dim=dim, page_size=page, lens=rng.randrange(1 << 20))
    if op == "append8":
        tokens = _log_int(rng, 1, 8192)
        batch = _log_int(rng, 1, min(64, tokens))
        new = max(1, tokens // batch)
        dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
        return dict(op=op, batch=batch, ctx_lo=1, ctx_hi=_log_int(rng, 16, 1000000), new_lo=rng.choice([1, new]),
                    new_hi=new, rot=rng.choice([dim, dim, dim // 2, 32]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.6, dtype=dtype, pad=rng.choice([0, 0, 11]), **sizes)
    batch = _log_int(rng, 1, 48)
    new = rng.choice([1, 1, min(_log_int(rng, 2, 256), max(1, 1024 // batch))])
    window = rng.choice([0, 0, 300 + new, 1024 + new]) if op == "attn8" else rng.choice([300 + new, 1024 + new, 4096])
    hi = _log_int(rng, 64, min(65536, 393216 // batch))
    # no more products than the largest listed case
    hi = max(64, min(hi, (4 * 256 * 32 * 8192) // (batch * new * hkv * group)))
    return dict(op=op, batch=batch, ctx_lo=rng.choice([1, max(1, hi // 8), hi]), ctx_hi=hi,
                new_lo=rng.choice([1, new]), new_hi=new, chain=new == 1 or rng.random() < 0.5, window=window,
                sinks=rng.choice([1, 4, 19, 128]) if window else 0, dtype=rng.choice(["f16", "bf16"]), **sizes)


# ---------------------------------------------------------------------------
# sizes of a case: the requests' lengths and trees, the same for every seed
# ---------------------------------------------------------------------------

def _lengths(case):
    """Per request: (cached tokens, new tokens, parents of the new tokens)."""
    rng = random.Random(1000003 * case["lens"] + case["batch"])
    reqs = []
    for _ in range(case["batch"]):
        ctx = _log_int(rng, case["ctx_lo"], case["ctx_hi"])
        new = rng.randint(case["new_lo"], case["new_hi"])
        # a drafted tree: mostly children of recent tokens, some siblings, now and then another root
        parents = [-1 if i == 0 or rng.random() < 0.04 else rng.randint(max(0, i - 9), i - 1) for i in range(new)]
        reqs.append((ctx, new, parents))
    return reqs


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _kept(case, ctx, new):
    """(tokens of the sinks, first token behind the gap) of what a request's new tokens can see."""
    if not case["window"]:
        return 0, 0
    first = max(0, ctx + 1 - case["window"])
    return min(case["sinks"], first), first


def work(case):
    if case["op"] == "append8":
        e, d, page = ESIZE[case["dtype"]], case["dim"], case["page_size"]
        tokens = sum(new for _, new, _ in _lengths(case))
        touched = sum((ctx + new - 1) // page - ctx // page + 1 for ctx, new, _ in _lengths(case))
        heads = case["hq"] + 2 * case["hkv"]
        moved = tokens * (d * (heads * e + case["hq"] * e + 2 * case["hkv"]) + 8) + 4 * touched * case["hkv"]
        rotated = case["hq"] + case["hkv"]
        flops = tokens * (rotated * (3 * case["rot"] + (4 * d if case["norm"] else 0)) + 4 * case["hkv"] * d)
        return {"bytes": moved + 2 * case["rot"] + (2 * d * e if case["norm"] else 0), "flops": flops}
    kv = pairs = tokens = pages = 0
    for ctx, new, parents in _lengths(case):
        sinks, first = _kept(case, ctx, new)
        kv += sinks + ctx + new - first
        pages += -(-sinks // case["page_size"]) + -(-(ctx + new - first) // case["page_size"])
        tokens += new
        pairs += new * (sinks + ctx - first)
        pairs += new * (new + 1) // 2 if case["chain"] else sum(_depths(parents)) + new
    e = ESIZE[case["dtype"]]
    moved = 2 * kv * case["hkv"] * case["dim"] * (1 if case["op"] == "attn8" else e)
    moved += tokens * case["hq"] * (2 * case["dim"] * e + 4) + 4 * pages + 16 * case["batch"]
    if case["op"] == "attn8":
        moved += 2 * pages * case["hkv"]
    if not case["chain"]:
        moved += tokens * 4 * _mask_words(case)
    return {"bytes": moved, "flops": 4 * case["dim"] * case["hq"] * pairs}


def _mask_words(case):
    return -(-case["new_hi"] // 32)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device=DEVICE)


def _prefix(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def _requests(case, seed):
    reqs = _lengths(case)
    random.Random(seed).shuffle(reqs)
    return reqs


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _cache8(gen, shape):
    """Codes and exponents of pages that hold values of about unit size."""
    codes = (_randn(gen, *shape) * 64.0).clamp(-CODE_MAX, CODE_MAX).to(CODE)
    exps = torch.randint(-7, -4, (shape[0], shape[2]), generator=gen, device=DEVICE).to(torch.int8)
    return codes, exps


def _prepare_append8(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, page = case["hq"], case["hkv"], case["dim"], case["page_size"]
    reqs = _requests(case, seed)
    # the pages that the new tokens lie on, of every request; what is cached before them is not touched
    touched = [(ctx + new - 1) // page - ctx // page + 1 for ctx, new, _ in reqs]
    pages = sum(touched) + max(4, sum(touched) // 4)
    ids = torch.randperm(pages, generator=gen, device=DEVICE).cpu().tolist()
    slots, positions, base = [], [], 0
    for (ctx, new, _), n in zip(reqs, touched):
        first = ctx // page
        slots += [ids[base + x // page - first] * page + x % page for x in range(ctx, ctx + new)]
        positions += range(ctx, ctx + new)
        base += n
    t = len(slots) + case["pad"]
    # one packed projection output, q and k and v are views of its rows
    qkv = (_randn(gen, t, hq + 2 * hkv, d) * 1.7).to(dt)
    half = case["rot"] // 2
    inv_freq = torch.tensor([10000.0 ** (-j / half) for j in range(half)], dtype=torch.float32, device=DEVICE)
    weight = [(1.0 + 0.2 * _randn(gen, d)).to(dt) for _ in range(2)] if case["norm"] else [None, None]
    k_pool, k_exp = _cache8(gen, (pages, page, hkv, d))
    v_pool, v_exp = _cache8(gen, (pages, page, hkv, d))
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                positions=_i32(positions + [0] * case["pad"]), slots=_i32(slots + [-1] * case["pad"]),
                inv_freq=inv_freq, q_weight=weight[0], k_weight=weight[1], eps=1e-6, k_pool=k_pool, v_pool=v_pool,
                k_exp=k_exp, v_exp=v_exp, q_out=torch.zeros(t, hq, d, dtype=dt, device=DEVICE))


def _prepare_attention(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt, page = DTYPES[case["dtype"]], case["page_size"]
    reqs = _requests(case, seed)
    counts = [-(-(ctx + new) // page) for ctx, new, _ in reqs]
    # pages whose tokens nobody sees any more were given back: the table's entries are -1, the pool holds the others
    kept = []
    for (ctx, new, _), n in zip(reqs, counts):
        sinks, first = _kept(case, ctx, new)
        kept += [p * page < sinks or (p + 1) * page > first for p in range(n)]
    live = sum(kept)
    pool_pages = live + max(4, live // 8)
    ids = iter(torch.randperm(pool_pages, generator=gen, device=DEVICE).cpu().tolist())
    indices = _i32(next(ids) if k else -1 for k in kept)
    tokens = sum(n for _, n, _ in reqs)
    words = _mask_words(case)
    mask, positions = None, []
    rows = []
    for ctx, new, parents in reqs:
        positions += range(ctx, ctx + new) if case["chain"] else [ctx + d for d in _depths(parents)]
        bits = []
        for i, p in enumerate(parents):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        rows += [[(b >> 32 * w & 0xFFFFFFFF) - (b >> 32 * w + 31 & 1) * (1 << 32) for w in range(words)] for b in bits]
    if not case["chain"]:
        mask = torch.tensor(rows, dtype=torch.int32, device=DEVICE)
    shape = (pool_pages, page, case["hkv"], case["dim"])
    state = dict(case=case, scale=case["dim"] ** -0.5,
                 q=(1.5 * _randn(gen, tokens, case["hq"], case["dim"])).to(dt), indices=indices,
                 indptr=_i32(_prefix(counts)), last_page_len=_i32((c + n - 1) % page + 1 for c, n, _ in reqs),
                 first_page_offset=_i32([0] * case["batch"]), qo_indptr=_i32(_prefix(n for _, n, _ in reqs)),
                 tree_mask=mask, positions=_i32(positions),
                 host=dict(total=[c + n for c, n, _ in reqs], new=[n for _, n, _ in reqs]))
    if case["op"] == "attn8":
        state["k_pool"], state["k_exp"] = _cache8(gen, shape)
        state["v_pool"], state["v_exp"] = _cache8(gen, shape)
    else:
        state["k_pool"], state["v_pool"] = _randn(gen, *shape).to(dt), _randn(gen, *shape).to(dt)
    return state


def prepare(case, seed):
    state = (_prepare_append8 if case["op"] == "append8" else _prepare_attention)(case, seed)
    if own:
        from paged_attention_decode_gb300 import pa_v2 as pa

        state["pa"] = pa
        if case["op"] != "append8":
            q = state["q"]
            sizes = (q.shape[0], case["batch"], case["hq"], case["hkv"], case["dim"])
            make = pa.attention_fp8_workspace if case["op"] == "attn8" else pa.tree_attention_workspace
            state["out"] = torch.empty_like(q)
            state["lse2"] = torch.empty(q.shape[:2], dtype=torch.float32, device=DEVICE)
            state["workspace"] = make(*sizes, device=q.device)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _own_append8, "attn8": _own_attn8, "sink16": _own_sink16}[op](state)
    return _plain_append8(state) if op == "append8" else _plain_attention(state)


def _own_append8(s):
    s["pa"].pa_v2_qk_rope_append_fp8(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_pool"],
                                     s["v_pool"], s["k_exp"], s["v_exp"], q_out=s["q_out"], q_weight=s["q_weight"],
                                     k_weight=s["k_weight"], eps=s["eps"], interleaved=s["case"]["interleaved"])
    return [s["q_out"], s["k_pool"], s["v_pool"], s["k_exp"], s["v_exp"]]


def _own_attn8(s):
    return list(s["pa"].pa_v2_attention_fp8(
        s["q"], s["k_pool"], s["v_pool"], s["k_exp"], s["v_exp"], s["indices"], s["indptr"], s["last_page_len"],
        s["first_page_offset"], s["qo_indptr"], s["scale"], tree_mask=s["tree_mask"], positions=s["positions"],
        sliding_window=s["case"]["window"], sinks=s["case"]["sinks"], out=s["out"], lse2_out=s["lse2"],
        workspace=s["workspace"]))


def _own_sink16(s):
    return list(s["pa"].pa_v2_tree_attention(
        s["q"], s["k_pool"], s["v_pool"], s["indices"], s["indptr"], s["last_page_len"], s["first_page_offset"],
        s["qo_indptr"], s["scale"], tree_mask=s["tree_mask"], positions=s["positions"],
        sliding_window=s["case"]["window"], sinks=s["case"]["sinks"], out=s["out"], lse2_out=s["lse2"],
        workspace=s["workspace"]))


def _plain_append8(s):
    case = s["case"]
    rot, half, page = case["rot"], case["rot"] // 2, case["page_size"]
    # in 64 bits: angles of far positions, and values next to a border between two codes
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = torch.cos(angle)[:, None, :], torch.sin(angle)[:, None, :]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.double()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((y, x[..., rot:]), -1)

    def into(pool, exps, x):
        pages = pool.shape[0]
        # padded tokens go to one more page behind the pool's, which is dropped
        slot = torch.where(s["slots"] < 0, pages * page, s["slots"]).long()
        at, entry = slot // page, slot % page
        top = torch.zeros(pages + 1, x.shape[1], dtype=x.dtype, device=x.device)
        top.index_reduce_(0, at, x.abs().amax(-1), "amax")
        first = torch.full((pages + 1,), page, dtype=torch.long, device=x.device)
        first.index_reduce_(0, at, entry, "amin")
        # the least exponent whose largest code holds the new tokens: top = m 2^e, 448 = 7/8 2^9
        m, e = torch.frexp(top)
        need = torch.where(m > 0.875, e - 8, e - 9)
        need = torch.where(top > 0, need, EXP_LO).clamp(EXP_LO, EXP_HI)[:pages]
        first = first[:pages, None]
        old = exps.long()
        new = torch.where(first == 0, need, torch.where(first < page, torch.maximum(old, need), old))
        # earlier tokens of a page whose exponent grew
        wide = pool.float()
        grown = (torch.arange(page, device=x.device)[None, :, None] < first[:, :, None]) & (first < page)[:, :, None]
        wide = torch.where(grown[..., None], torch.ldexp(wide, (old - new)[:, None, :, None]), wide)
        flat = torch.cat((wide, torch.zeros_like(wide[:1]))).flatten(0, 1)
        scale = torch.cat((new, torch.zeros_like(new[:1])))[at][..., None]
        flat[slot] = torch.ldexp(x, -scale).clamp(-CODE_MAX, CODE_MAX).float()
        pool.copy_(flat[:pages * page].view(wide.shape).to(CODE))
        exps.copy_(new)

    live = (s["slots"] >= 0)[:, None, None]
    s["q_out"].copy_(torch.where(live, turned(s["q"], s["q_weight"]), s["q_out"].double()))
    into(s["k_pool"], s["k_exp"], turned(s["k"], s["k_weight"]))
    into(s["v_pool"], s["v_exp"], s["v"].double())
    return [s["q_out"], s["k_pool"], s["v_pool"], s["k_exp"], s["v_exp"]]


def _plain_attention(s):
    case = s["case"]
    page, hkv, dim, window = case["page_size"], case["hkv"], case["dim"], case["window"]
    group, dev, batch = case["hq"] // hkv, s["q"].device, case["batch"]
    pages = (s["indptr"][1:] - s["indptr"][:-1]).long()
    total = (pages - 1) * page + s["last_page_len"].long()
    new = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    ctx = total - new
    # the keys that any new token sees, padded to the most: the sinks, then all from the first token's window on
    first = (ctx + 1 - window).clamp(min=0) if window else torch.zeros_like(ctx)
    sinks = first.clamp(max=case["sinks"])
    longest = max(t - f + k for t, (k, f) in
                  zip(s["host"]["total"], (_kept(case, t - n, n) for t, n in zip(s["host"]["total"], s["host"]["new"]))))
    j = torch.arange(longest, device=dev)[None, :]
    key = torch.where(j < sinks[:, None], j, first[:, None] + j - sinks[:, None])           # [batch, keys]
    live = key < total[:, None]
    key = torch.minimum(key, total[:, None] - 1)
    ids = s["indices"].long()[s["indptr"][:-1].long()[:, None] + key // page].clamp(min=0)

    def rows(pool, exps):
        x = pool[ids, key % page].float()                                                   # [batch, keys, hkv, dim]
        return x if exps is None else torch.ldexp(x, exps[ids][..., None])

    k, v = rows(s["k_pool"], s.get("k_exp")), rows(s["v_pool"], s.get("v_exp"))
    most = max(s["host"]["new"])
    i = torch.arange(most, device=dev)[None, :]
    token = torch.minimum(s["qo_indptr"][:-1].long()[:, None] + i, s["qo_indptr"][-1].long() - 1)  # [batch, most]
    q = s["q"][token].float().reshape(batch, most, hkv, group, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    at = s["positions"].long()[token][..., None]                                            # the token's own position
    far, draft = key[:, None, :], (key - ctx[:, None])[:, None, :]                          # draft: new token's number
    seen = (far < case["sinks"]) | (far > at - window) if window else torch.ones_like(far, dtype=torch.bool)
    if case["chain"]:
        seen = seen & (far <= at)
    else:
        word = s["tree_mask"].long()[token].gather(2, (draft // 32).clamp(0, s["tree_mask"].shape[1] - 1)
                                                   .expand(-1, most, -1))
        seen = torch.where(draft < 0, seen, (word >> (draft.clamp(min=0) % 32)) & 1 == 1)
    seen = (seen & live[:, None, :])[:, None, :, None, :]
    score = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    score = torch.where(seen, score.view(batch, hkv, most, group, -1), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    norm = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).view(batch, hkv, most, group, dim) / norm
    lse = (top + torch.log(norm))[..., 0] / math.log(2.0)
    # the tokens packed again
    t = torch.arange(s["q"].shape[0], device=dev)
    r = torch.searchsorted(s["qo_indptr"][1:].long(), t, right=True)
    i = t - s["qo_indptr"].long()[r]
    o, lse = o.permute(0, 2, 1, 3, 4).flatten(2, 3), lse.permute(0, 2, 1, 3).flatten(2, 3)
    return [o[r, i].to(s["q"].dtype), lse[r, i]]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "append8":
        return _exact_append8(_prepare_append8(case, seed))
    return _exact_attention(_prepare_attention(case, seed))


def _exact_append8(s):
    """The 8-bit outputs are given before their rounding: what the codes approximate, in units of 2^exponent."""
    case = s["case"]
    half, page, hkv = case["rot"] // 2, case["page_size"], case["hkv"]
    turn = s["positions"].double().reshape(-1, 1, 1) * s["inv_freq"].double()
    turn = torch.complex(torch.cos(turn), torch.sin(turn))
    one = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
    two = one + (1 if case["interleaved"] else half)

    def done(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt() * weight.double()
        z = torch.complex(x[..., one], x[..., two]) * turn
        x = x.clone()
        x[..., one], x[..., two] = z.real, z.imag
        return x

    q = s["q_out"].double()
    slots = s["slots"].tolist()
    count = sum(x >= 0 for x in slots)
    q[:count] = done(s["q"], s["q_weight"])[:count]
    runs = []                                   # (first token, behind the last, page) of the tokens on one page
    for t, slot in enumerate(slots[:count]):
        if runs and runs[-1][2] == slot // page:
            runs[-1][1] = t + 1
        else:
            runs.append([t, t + 1, slot // page])
    out = []
    for pool, exps, x in ((s["k_pool"], s["k_exp"], done(s["k"], s["k_weight"])), (s["v_pool"], s["v_exp"], s["v"].double())):
        wide, exps = pool.double(), exps.cpu().long()
        tops = x.abs().amax(-1).cpu().tolist()
        grow = torch.zeros(exps.shape, dtype=torch.float64)
        before = torch.zeros(exps.shape[0], dtype=torch.long)
        for t0, t1, p in runs:
            before[p] = slots[t0] % page
            for h in range(hkv):
                top, e = max(tops[t][h] for t in range(t0, t1)), EXP_LO
                while e < EXP_HI and top > CODE_MAX * 2.0 ** e:
                    e += 1
                old = int(exps[p, h])
                exps[p, h] = e if slots[t0] % page == 0 else max(e, old)
                grow[p, h] = old - int(exps[p, h])
        earlier = torch.arange(page)[None, :] < before[:, None]
        factor = torch.where(earlier[:, :, None], torch.exp2(grow)[:, None, :], 1.0)
        wide *= factor.to(DEVICE)[..., None]
        at = s["slots"][:count].long()
        unit = torch.exp2(exps.double()).to(DEVICE)[at // page][..., None]
        wide.flatten(0, 1)[at] = (x[:count] / unit).clamp(-CODE_MAX, CODE_MAX)
        out.append((wide, exps))
    return [q, out[0][0], out[1][0], out[0][1], out[1][1]]


def _exact_attention(s):
    case = s["case"]
    page, hkv, window = case["page_size"], case["hkv"], case["window"]
    group = case["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse2 = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    indptr, starts, lpl = s["indptr"].tolist(), s["qo_indptr"].tolist(), s["last_page_len"].tolist()
    for r in range(case["batch"]):
        ids = s["indices"][indptr[r]:indptr[r + 1]].long()
        length = (len(ids) - 1) * page + lpl[r]
        t0, t1 = starts[r], starts[r + 1]
        cached = length - (t1 - t0)
        where = s["positions"][t0:t1].long()
        y = torch.arange(length, device=DEVICE)
        bias = torch.zeros(t1 - t0, length, dtype=torch.float64, device=DEVICE)
        if window:
            hidden = (y[None, :] >= case["sinks"]) & (where[:, None] - y[None, :] >= window)
            bias[hidden] = -math.inf
        for n in range(t1 - t0):
            if case["chain"]:
                bias[:n, cached + n] = -math.inf
            else:
                sees = (s["tree_mask"][t0:t1, n // 32].long() >> n % 32) % 2 != 0
                bias[:, cached + n] = torch.where(sees, 0.0, -math.inf)
        some = (bias > -math.inf).any(0).nonzero()[:, 0]        # the rows of given-back pages are not read
        bias = bias[:, some]
        pg, row = ids[some // page], some % page
        for h in range(hkv):
            k, v = s["k_pool"][pg, row, h].double(), s["v_pool"][pg, row, h].double()
            if case["op"] == "attn8":
                k = k * torch.exp2(s["k_exp"][pg, h].double())[:, None]
                v = v * torch.exp2(s["v_exp"][pg, h].double())[:, None]
            for g in range(group):
                head = h * group + g
                score = s["q"][t0:t1, head].double() @ k.T * s["scale"] + bias
                norm = torch.logsumexp(score, 1)
                out[t0:t1, head] = torch.exp(score - norm[:, None]) @ v
                lse2[t0:t1, head] = norm / math.log(2.0)
    return [out, lse2]
