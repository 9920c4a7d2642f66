"""Measured cases of the step operators: table building, q/k norm + rotation + cache append, tree attention.

Each case is one pass through one operator of a serving step over a paged KV cache:

- ``tables``: page table, slot map, positions and tree masks of a step from the requests' lengths;
- ``qk``: per-head norm of q and k, position rotation, and the append of k and v to the pools;
- ``tree``: attention of every request's drafted tokens (a tree or a chain) over its cached pages.

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
DEVICE = "cuda"


def listed():
    return [
        # tables of one speculative step: 32 requests, trees of up to 64 drafted tokens, new pages handed out
        dict(name="tables_tree_b32", op="tables", batch=32, ctx_lo=512, ctx_hi=8192, new_lo=1, new_hi=64,
             tree=True, page_size=16, window=0, spare_tokens=0, lens=1),
        # the largest: one new token each for 512 long requests, a padded token capacity
        dict(name="tables_decode_b512", op="tables", batch=512, ctx_lo=4096, ctx_hi=131072, new_lo=1, new_hi=1,
             tree=False, page_size=16, window=0, spare_tokens=128, lens=2),
        # single-token decode of a small batch: rotation only, q in f32 for the decode call
        dict(name="qk_decode_b8", op="qk", tokens=8, hq=32, hkv=8, dim=128, rot=128, interleaved=False, norm=False,
             dtype="f16", q32=True, page_size=16, pos_hi=32768),
        # 32 trees of 64 drafted tokens to verify
        dict(name="qk_verify_2048", op="qk", tokens=2048, hq=32, hkv=8, dim=128, rot=128, interleaved=False,
             norm=True, dtype="bf16", q32=False, page_size=16, pos_hi=131072),
        # a prompt's chunk
        dict(name="qk_prompt_16384", op="qk", tokens=16384, hq=32, hkv=8, dim=128, rot=128, interleaved=False,
             norm=True, dtype="bf16", q32=False, page_size=16, pos_hi=131072),
        # an f32 cache with a partial, interleaved rotation, few heads and an odd page size
        dict(name="qk_odd_f32", op="qk", tokens=777, hq=12, hkv=4, dim=64, rot=32, interleaved=True, norm=True,
             dtype="f32", q32=True, page_size=5, pos_hi=1000000),
        # the smallest attention call: a small tree over a short context, latency bound
        dict(name="tree_b1_8tok_1k", op="tree", batch=1, ctx_lo=1024, ctx_hi=1024, new_lo=8, new_hi=8, chain=False,
             hq=32, hkv=8, dim=128, page_size=16, window=0, dtype="f16", lens=3),
        # one long request with a full tree: the 32K decode shape, 64 drafted tokens
        dict(name="tree_b1_64tok_32k", op="tree", batch=1, ctx_lo=32768, ctx_hi=32768, new_lo=64, new_hi=64,
             chain=False, hq=32, hkv=8, dim=128, page_size=16, window=0, dtype="f16", lens=4),
        # a ragged serving batch with trees of different sizes
        dict(name="tree_b16_ragged", op="tree", batch=16, ctx_lo=1024, ctx_hi=16384, new_lo=1, new_hi=64,
             chain=False, hq=32, hkv=8, dim=128, page_size=16, window=0, dtype="bf16", lens=5),
        # chain verification (four drafted tokens and the last accepted one) under a sliding window
        dict(name="chain_b32_5tok_window", op="tree", batch=32, ctx_lo=512, ctx_hi=16384, new_lo=5, new_hi=5,
             chain=True, hq=32, hkv=8, dim=128, page_size=16, window=4096, dtype="bf16", lens=6),
        # the largest: wide trees over long contexts, bound by the tensor cores
        dict(name="tree_b4_256tok_32k", op="tree", batch=4, ctx_lo=32768, ctx_hi=32768, new_lo=256, new_hi=256,
             chain=False, hq=32, hkv=8, dim=128, page_size=16, window=0, dtype="bf16", lens=7),
        # odd everything: page size 5, three query heads per KV head, head_dim 64, short ragged contexts
        dict(name="tree_b7_odd", op="tree", batch=7, ctx_lo=33, ctx_hi=2999, new_lo=1, new_hi=33, chain=False,
             hq=24, hkv=8, dim=64, page_size=5, window=0, dtype="f16", lens=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "qk", "tree", "tree"])
    if op == "tables":
        page = rng.choice([1, 3, 8, 16, 16, 64])
        batch = _log_int(rng, 1, 512)
        hi = _log_int(rng, 64, min(131072, 512 * 8192 * page // batch))
        new = rng.choice([1, 5, _log_int(rng, 1, 200)])
        return dict(op="tables", batch=batch, ctx_lo=min(hi, rng.choice([1, 100, 1024])), ctx_hi=hi, new_lo=1,
                    new_hi=min(new, 20000 // batch + 1), tree=rng.random() < 0.5, page_size=page,
                    window=rng.choice([0, 0, 300, 4096]), spare_tokens=rng.choice([0, 0, 37]),
                    lens=rng.randrange(1 << 20))
    if op == "qk":
        dim = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 3, 4, 7, 8])
        if hkv * group > 40:
            group = 4
        dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
        return dict(op="qk", tokens=_log_int(rng, 1, 8192), hq=hkv * group, hkv=hkv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 32]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.6, dtype=dtype, q32=dtype == "f32" or rng.random() < 0.4,
                    page_size=rng.choice([1, 5, 16, 16, 64]), pos_hi=_log_int(rng, 64, 1000000))
    hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 3, 4, 4, 7, 8])
    if hkv * group > 40:
        group = 4
    batch = _log_int(rng, 1, 48)
    new = min(_log_int(rng, 1, 256), max(1, 1024 // batch))
    hi = _log_int(rng, 64, min(65536, 393216 // batch))
    # no more products than the largest listed case
    hi = max(64, min(hi, (4 * 256 * 32 * 32768) // (batch * new * hkv * group)))
    chain = rng.random() < 0.4
    return dict(op="tree", batch=batch, ctx_lo=rng.choice([1, max(1, hi // 8), hi]), ctx_hi=hi,
                new_lo=rng.choice([1, new]), new_hi=new, chain=chain, hq=hkv * group, hkv=hkv,
                dim=rng.choice([64, 128, 128]), page_size=rng.choice([1, 5, 8, 16, 16, 16, 48, 64]),
                window=rng.choice([0, 0, 0, 1024 + new]), dtype=rng.choice(["f16", "bf16"]),
                lens=rng.randrange(1 << 20))


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


def _visible(case, ctx, new):
    total = ctx + new
    return min(total, case["window"]) if case["window"] else total


def work(case):
    if case["op"] == "tables":
        page = case["page_size"]
        read = wrote = 0
        for ctx, new, _ in _lengths(case):
            total = ctx + new
            seen = _visible(case, ctx, new)
            pages = -(-total // page) - (total - seen) // page
            taken = -(-total // page) - -(-ctx // page)
            read += 8 + 4 * pages + (4 * new if case["tree"] else 0)
            wrote += 16 + 4 * pages + 4 * taken + 8 * new
            if case["tree"]:
                wrote += new * 4 * _mask_words(case)
        return {"bytes": read + wrote + 8 * case["spare_tokens"] + 12, "flops": 0}
    if case["op"] == "qk":
        e, t, d = ESIZE[case["dtype"]], case["tokens"], case["dim"]
        heads = case["hq"] + 2 * case["hkv"]
        q_out = 4 if case["q32"] else e
        moved = t * d * (heads * e + case["hq"] * q_out + 2 * case["hkv"] * e) + 8 * t + 2 * case["rot"]
        rotated = case["hq"] + case["hkv"]
        flops = t * rotated * (3 * case["rot"] + (4 * d if case["norm"] else 0))
        return {"bytes": moved + (2 * d * e if case["norm"] else 0), "flops": flops}
    kv = pairs = tokens = 0
    for ctx, new, parents in _lengths(case):
        seen = _visible(case, ctx, new)
        kv += seen
        tokens += new
        pairs += new * (seen - new)
        pairs += new * (new + 1) // 2 if case["chain"] else sum(_depths(parents)) + new
    e = ESIZE[case["dtype"]]
    moved = 2 * kv * case["hkv"] * case["dim"] * e + tokens * case["hq"] * (2 * case["dim"] * e + 4)
    pages = kv // case["page_size"] * 4 + 16 * case["batch"]
    mask = 0 if case["chain"] else tokens * 4 * _mask_words(case)
    return {"bytes": moved + pages + mask, "flops": 4 * case["dim"] * case["hq"] * pairs}


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


def _prepare_tables(case, seed):
    page, batch = case["page_size"], case["batch"]
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    reqs = _requests(case, seed)
    width = -(-(case["ctx_hi"] + case["new_hi"]) // page)
    tokens = sum(n for _, n, _ in reqs) + case["spare_tokens"]
    listed_pages = taken = 0
    for ctx, new, _ in reqs:
        listed_pages += -(-(ctx + new) // page)
        taken += -(-(ctx + new) // page) - -(-ctx // page)
    ids = torch.randperm(batch * width + taken + 16, generator=gen, device=DEVICE).to(torch.int32)
    parents = [p for _, _, ps in reqs for p in ps] + [-1] * case["spare_tokens"]
    words = _mask_words(case) if case["tree"] else 0
    return dict(
        case=case, cached=_i32(c for c, _, _ in reqs), new=_i32(n for _, n, _ in reqs),
        block_table=ids[:batch * width].reshape(batch, width).clone(), free=ids[batch * width:].clone(),
        parents=_i32(parents) if case["tree"] else None, longest=max(n for _, n, _ in reqs),
        indptr=_i32([0] * (batch + 1)), indices=_i32([-1] * (listed_pages + 8)), last_page_len=_i32([0] * batch),
        first_page_offset=_i32([0] * batch), qo_indptr=_i32([0] * (batch + 1)), slots=_i32([0] * tokens),
        positions=_i32([0] * tokens), tree_mask=torch.zeros(tokens, words, dtype=torch.int32, device=DEVICE),
        pages_needed=_i32([0]))


def _prepare_qk(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    t, hq, hkv, d, page = case["tokens"], case["hq"], case["hkv"], case["dim"], case["page_size"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32)

    # one packed projection output, q and k and v are views of its rows
    qkv = (randn(t, hq + 2 * hkv, d) * 1.7).to(dt)
    pages = -(-(t + t // 2 + 16) // page)
    rows = torch.randperm(pages * page, generator=gen, device=DEVICE)[:t].to(torch.int32)
    positions = torch.randint(0, case["pos_hi"], (t,), generator=gen, device=DEVICE).to(torch.int32)
    half = case["rot"] // 2
    inv_freq = torch.tensor([10000.0 ** (-j / half) for j in range(half)], dtype=torch.float32, device=DEVICE)
    weight = [(1.0 + 0.2 * randn(d)).to(dt) for _ in range(2)] if case["norm"] else [None, None]
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], positions=positions, slots=rows,
                inv_freq=inv_freq, q_weight=weight[0], k_weight=weight[1], eps=1e-6,
                k_pool=randn(pages, page, hkv, d).to(dt), v_pool=randn(pages, page, hkv, d).to(dt),
                q_out=torch.zeros(t, hq, d, dtype=torch.float32 if case["q32"] else dt, device=DEVICE))


def _prepare_tree(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    dt, page = DTYPES[case["dtype"]], case["page_size"]
    reqs = _requests(case, seed)
    pages, lpl, fpo, seen_all = [], [], [], []
    for ctx, new, _ in reqs:
        total = ctx + new
        seen = _visible(case, ctx, new)
        first = total - seen
        pages.append(-(-total // page) - first // page)
        lpl.append((total - 1) % page + 1)
        fpo.append(first % page)
        seen_all.append(seen)
    pool_pages = sum(pages) + max(4, sum(pages) // 8)
    shape = (pool_pages, page, case["hkv"], case["dim"])

    def randn(*size):
        return torch.randn(*size, generator=gen, device=DEVICE, dtype=torch.float32)

    tokens = sum(n for _, n, _ in reqs)
    words = _mask_words(case)
    mask = None
    if not case["chain"]:
        rows = []
        for _, _, parents in reqs:
            bits = []
            for i, p in enumerate(parents):
                bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            rows += [[(b >> 32 * w & 0xFFFFFFFF) - (b >> 32 * w + 31 & 1) * (1 << 32) for w in range(words)]
                     for b in bits]
        mask = torch.tensor(rows, dtype=torch.int32, device=DEVICE)
    return dict(case=case, scale=case["dim"] ** -0.5, q=(1.5 * randn(tokens, case["hq"], case["dim"])).to(dt),
                k_pool=randn(*shape).to(dt), v_pool=randn(*shape).to(dt),
                indices=torch.randperm(pool_pages, generator=gen, device=DEVICE)[:sum(pages)].to(torch.int32),
                indptr=_i32(_prefix(pages)), last_page_len=_i32(lpl), first_page_offset=_i32(fpo),
                qo_indptr=_i32(_prefix(n for _, n, _ in reqs)), tree_mask=mask,
                host=dict(pages=_prefix(pages), tokens=_prefix(n for _, n, _ in reqs), seen=seen_all, fpo=fpo))


def prepare(case, seed):
    state = {"tables": _prepare_tables, "qk": _prepare_qk, "tree": _prepare_tree}[case["op"]](case, seed)
    if own:
        from paged_attention_decode_gb300 import pa_v2 as pa

        state["pa"] = pa
        if case["op"] == "tables":
            state["tables"] = pa.StepTables(*(state[k] for k in TABLE_FIELDS))
            if not case["tree"]:
                state["tables"].tree_mask = None
        if case["op"] == "tree":
            q, pool = state["q"], state["k_pool"]
            state["out"] = torch.empty_like(q)
            state["lse2"] = torch.empty(q.shape[:2], dtype=torch.float32, device=DEVICE)
            state["workspace"] = pa.tree_attention_workspace(q.shape[0], case["batch"], case["hq"], case["hkv"],
                                                             case["dim"], device=q.device)
    return state


TABLE_FIELDS = ("indptr", "indices", "last_page_len", "first_page_offset", "qo_indptr", "slots", "positions",
                "tree_mask", "pages_needed")


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "qk": _own_qk, "tree": _own_tree}[op](state)
    return {"tables": _plain_tables, "qk": _plain_qk, "tree": _plain_tree}[op](state)


def _own_tables(s):
    case = s["case"]
    s["pa"].pa_v2_build_tables(s["cached"], s["new"], s["block_table"], case["page_size"], s["tables"],
                               free_pages=s["free"], parents=s["parents"], window=case["window"])
    return [s["block_table"]] + [s[k] for k in TABLE_FIELDS]


def _own_qk(s):
    s["pa"].pa_v2_qk_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_pool"],
                                 s["v_pool"], q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                 eps=s["eps"], interleaved=s["case"]["interleaved"])
    return [s["q_out"], s["k_pool"], s["v_pool"]]


def _own_tree(s):
    out, lse2 = s["pa"].pa_v2_tree_attention(
        s["q"], s["k_pool"], s["v_pool"], s["indices"], s["indptr"], s["last_page_len"], s["first_page_offset"],
        s["qo_indptr"], s["scale"], tree_mask=s["tree_mask"], out=s["out"], lse2_out=s["lse2"],
        workspace=s["workspace"])
    return [out, lse2]


def _plain_tables(s):
    case = s["case"]
    page, dev = case["page_size"], s["cached"].device
    cached, new, table = s["cached"].long(), s["new"].long(), s["block_table"]
    total = cached + new
    have, need = (cached + page - 1) // page, (total + page - 1) // page
    take = need - have
    first_free = torch.cumsum(take, 0) - take
    col = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    source = (first_free[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][source], table))
    seen = total.clamp(max=case["window"]) if case["window"] else total
    start = total - seen
    p0 = start // page
    pages = need - p0
    s["indptr"][1:] = torch.cumsum(pages, 0)
    s["last_page_len"].copy_(torch.where(pages > 0, (total - 1) % page + 1, 0))
    s["first_page_offset"].copy_(torch.where(pages > 0, start % page, 0))
    s["qo_indptr"][1:] = torch.cumsum(new, 0)
    s["pages_needed"].copy_(take.sum())
    at = torch.arange(s["indices"].numel(), device=dev)
    ends = s["indptr"][1:].long()
    r = torch.searchsorted(ends, at, right=True).clamp(max=case["batch"] - 1)
    src = (p0[r] + at - s["indptr"].long()[r]).clamp(0, table.shape[1] - 1)
    s["indices"].copy_(torch.where(at < ends[-1], table[r, src], s["indices"]))
    at = torch.arange(s["slots"].numel(), device=dev)
    live = at < s["qo_indptr"][-1]
    r = torch.searchsorted(s["qo_indptr"][1:].long(), at, right=True).clamp(max=case["batch"] - 1)
    base = s["qo_indptr"].long()[r]
    i = at - base
    pos = cached[r] + i
    slot = table[r, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    s["slots"].copy_(torch.where(live, slot, -1))
    if case["tree"]:
        words = s["tree_mask"].shape[1]
        reach = i[:, None] == torch.arange(32 * words, device=dev)[None, :]
        jump = torch.where(live & (s["parents"] >= 0), base + s["parents"], -1)
        hops = 1
        while hops < s["longest"]:
            reach = reach | (reach[jump.clamp(min=0)] & (jump >= 0)[:, None])
            jump = torch.where(jump >= 0, jump[jump.clamp(min=0)], -1)
            hops *= 2
        bits = (reach.long().reshape(-1, words, 32) << torch.arange(32, device=dev)).sum(-1)
        bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits)
        s["tree_mask"].copy_(torch.where(live[:, None], bits, s["tree_mask"]))
        pos = cached[r] + reach.sum(-1) - 1
    s["positions"].copy_(torch.where(live, pos, 0))
    return [table] + [s[k] for k in TABLE_FIELDS]


def _plain_qk(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2

    def normed(x, weight):
        x = x.float()
        if weight is None:
            return x
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()

    # angles of far positions need 64 bits: 1e6 radians in 32 are off by several hundredths
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def rotated(x):
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned, x[..., rot:]), -1)

    s["q_out"].copy_(rotated(normed(s["q"], s["q_weight"])))
    rows = s["slots"].long()
    k_rows, v_rows = s["k_pool"].flatten(0, 1), s["v_pool"].flatten(0, 1)
    k_rows[rows] = rotated(normed(s["k"], s["k_weight"])).to(k_rows.dtype)
    v_rows[rows] = s["v"]
    return [s["q_out"], s["k_pool"], s["v_pool"]]


def _plain_tree(s):
    case, host = s["case"], s["host"]
    page, hkv, dim = case["page_size"], case["hkv"], case["dim"]
    group = case["hq"] // hkv
    dev = s["q"].device
    outs, lses = [], []
    for r in range(case["batch"]):
        t0, t1, seen = host["tokens"][r], host["tokens"][r + 1], host["seen"][r]
        n = t1 - t0
        entry = host["fpo"][r] + torch.arange(seen, device=dev)
        ids = s["indices"][host["pages"][r]:host["pages"][r + 1]].long()
        rows = ids[entry // page] * page + entry % page
        k = s["k_pool"].flatten(0, 1)[rows].float().permute(1, 2, 0)            # [hkv, dim, seen]
        v = s["v_pool"].flatten(0, 1)[rows].float().permute(1, 0, 2)            # [hkv, seen, dim]
        q = s["q"][t0:t1].float().reshape(n, hkv, group, dim).permute(1, 0, 2, 3).reshape(hkv, n * group, dim)
        draft = torch.arange(n, device=dev)
        if case["chain"]:
            allowed = draft[None, :] <= draft[:, None]
        else:
            allowed = (s["tree_mask"][t0:t1][:, draft // 32] >> (draft % 32)) & 1 == 1
        score = torch.bmm(q, k) * s["scale"]
        tail = score.view(hkv, n, group, seen)[..., seen - n:]
        tail.masked_fill_(~allowed[None, :, None, :], -math.inf)
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        o = torch.bmm(p, v) / total
        outs.append(o.view(hkv, n, group, dim).permute(1, 0, 2, 3).reshape(n, hkv * group, dim))
        lse = (top + torch.log(total)) / math.log(2.0)
        lses.append(lse.view(hkv, n, group).permute(1, 0, 2).reshape(n, hkv * group))
    return [torch.cat(outs).to(s["q"].dtype), torch.cat(lses)]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return _exact_tables(case, seed)
    if case["op"] == "qk":
        return _exact_qk(_prepare_qk(case, seed))
    return _exact_tree(_prepare_tree(case, seed))


def _exact_tables(case, seed):
    s = _prepare_tables(case, seed)
    page = case["page_size"]
    out = {k: s[k].cpu().long() for k in TABLE_FIELDS}
    table, free = s["block_table"].cpu().long(), s["free"].cpu().long()
    next_free = next_index = next_token = 0
    for r, (ctx, new, parents) in enumerate(_requests(case, seed)):
        total = ctx + new
        while -(-ctx // page) < -(-total // page):      # one more page for the new tokens
            table[r, -(-ctx // page)] = free[next_free]
            next_free += 1
            ctx = min(total, (-(-ctx // page) + 1) * page)
        ctx = total - new
        first = max(0, total - case["window"]) if case["window"] else 0
        ids = table[r, first // page:(total - 1) // page + 1]
        out["indices"][next_index:next_index + len(ids)] = ids
        next_index += len(ids)
        out["indptr"][r + 1] = next_index
        out["last_page_len"][r] = (total - 1) % page + 1
        out["first_page_offset"][r] = first % page
        for i in range(new):
            at, up = ctx + i, i
            depth, line = 0, [i]
            while case["tree"] and parents[up] >= 0:
                up = parents[up]
                line.append(up)
                depth += 1
            out["slots"][next_token] = table[r, at // page] * page + at % page
            out["positions"][next_token] = ctx + (depth if case["tree"] else i)
            if case["tree"]:
                for w in range(out["tree_mask"].shape[1]):
                    bits = sum(1 << j % 32 for j in line if j // 32 == w)
                    out["tree_mask"][next_token, w] = bits - (1 << 32 if bits >> 31 else 0)
            next_token += 1
        out["qo_indptr"][r + 1] = next_token
    out["slots"][next_token:] = -1
    out["positions"][next_token:] = 0
    out["pages_needed"][0] = next_free
    return [table] + [out[k] for k in TABLE_FIELDS]


def _exact_qk(s):
    case = s["case"]
    half = case["rot"] // 2
    turn = s["positions"].double().reshape(-1, 1, 1) * s["inv_freq"].double()
    turn = torch.complex(torch.cos(turn), torch.sin(turn))
    if case["interleaved"]:
        first = torch.arange(half, device=DEVICE) * 2
        second = first + 1
    else:
        first = torch.arange(half, device=DEVICE)
        second = first + half

    def done(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt() * weight.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    pools = []
    for pool, rows in ((s["k_pool"], done(s["k"], s["k_weight"])), (s["v_pool"], s["v"].double())):
        wide = pool.double()
        flat = wide.view(-1, case["hkv"], case["dim"])
        flat.index_copy_(0, s["slots"].long(), rows)
        pools.append(wide)
    return [done(s["q"], s["q_weight"])] + pools


def _exact_tree(s):
    case = s["case"]
    page, hkv = case["page_size"], case["hkv"]
    group = case["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse2 = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEVICE)
    indptr, starts = s["indptr"].tolist(), s["qo_indptr"].tolist()
    fpo, lpl = s["first_page_offset"].tolist(), s["last_page_len"].tolist()
    for r in range(case["batch"]):
        ids = s["indices"][indptr[r]:indptr[r + 1]].long()
        last = (len(ids) - 1) * page + lpl[r]
        t0, t1 = starts[r], starts[r + 1]
        n = t1 - t0
        bias = torch.zeros(n, last - fpo[r], dtype=torch.float64, device=DEVICE)
        for j in range(n):
            if case["chain"]:
                sees = torch.arange(n, device=DEVICE) >= j
            else:
                sees = (s["tree_mask"][t0:t1, j // 32].long() >> j % 32) % 2 != 0
            bias[:, j - n] = torch.where(sees, 0.0, -math.inf)
        for h in range(hkv):
            k = s["k_pool"][ids, :, h].reshape(-1, case["dim"])[fpo[r]:last].double()
            v = s["v_pool"][ids, :, h].reshape(-1, case["dim"])[fpo[r]:last].double()
            for g in range(group):
                head = h * group + g
                score = s["q"][t0:t1, head].double() @ k.T * s["scale"] + bias
                norm = torch.logsumexp(score, 1)
                out[t0:t1, head] = torch.exp(score - norm[:, None]) @ v
                lse2[t0:t1, head] = norm / math.log(2.0)
    return [out, lse2]
