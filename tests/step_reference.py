"""Plain 64-bit references of the step operators (tables, q/k preparation, tree attention) for the tests.

Written from the definitions, on the CPU, element by element where that is affordable; they share nothing
with the library.  The tolerances count roundings: half a step of the type where a value is rounded to it
(``eps / 2``, relative), and the f32 arithmetic's worst case where sums are formed.
"""
from __future__ import annotations

import math
import random

import torch

LOG2E = 1.0 / math.log(2.0)


def random_tree(rng: random.Random, n: int, root_chance: float = 0.1) -> list[int]:
    return [-1 if i == 0 or rng.random() < root_chance else rng.randint(max(0, i - 6), i - 1) for i in range(n)]


def ancestors(parents: list[int] | None, i: int) -> list[int]:
    """Token i and its ancestors (a chain when parents is None), nearest first."""
    line = [i]
    while True:
        up = line[-1] - 1 if parents is None else parents[line[-1]]
        if up < 0:
            return line
        line.append(up)


def words_of(bits: int, words: int) -> list[int]:
    out = []
    for w in range(words):
        x = (bits >> (32 * w)) & 0xFFFFFFFF
        out.append(x - (1 << 32) if x >> 31 else x)
    return out


def tree_mask(parents_per_request, words: int) -> torch.Tensor:
    rows = []
    for parents in parents_per_request:
        for i in range(len(parents)):
            rows.append(words_of(sum(1 << j for j in ancestors(parents, i)), words))
    return torch.tensor(rows, dtype=torch.int32).reshape(-1, words)


def tables_ref(cached, new, block_table, free, parents, page_size, window, mask_words):
    """Lists of the step's tables: {field: list or tensor} with the valid parts only; block_table extended."""
    table = block_table.clone()
    out = dict(indptr=[0], indices=[], last_page_len=[], first_page_offset=[], qo_indptr=[0], slots=[], positions=[],
               tree_mask=[], pages_needed=0)
    for r, (c, n) in enumerate(zip(cached, new)):
        t = c + n
        for col in range(-(-c // page_size), -(-t // page_size)):
            if free is not None:
                table[r, col] = int(free[out["pages_needed"]])
                out["pages_needed"] += 1
        start = max(0, t - window) if window else 0
        pages = [int(table[r, col]) for col in range(start // page_size, -(-t // page_size))]
        out["indices"] += pages
        out["indptr"].append(len(out["indices"]))
        out["last_page_len"].append((t - 1) % page_size + 1 if t else 0)
        out["first_page_offset"].append(start % page_size if t else 0)
        tree = parents[r] if parents is not None else None
        for i in range(n):
            at = c + i
            out["slots"].append(int(table[r, at // page_size]) * page_size + at % page_size)
            line = ancestors(tree, i)
            out["positions"].append(c + len(line) - 1)
            if mask_words:
                out["tree_mask"].append(words_of(sum(1 << j for j in line), mask_words))
        out["qo_indptr"].append(out["qo_indptr"][-1] + n)
    out["block_table"] = table
    return out


def sliding_tables_ref(cached, new, block_table, free, parents, page_size, window, mask_words):
    """tables_ref for a model whose tokens each see a window of positions up to their own."""
    out = tables_ref(cached, new, block_table, free, parents, page_size, 0, mask_words)
    table = out["block_table"]
    out.update(indptr=[0], indices=[], first_page_offset=[], tree_mask=[])
    for r, (c, n) in enumerate(zip(cached, new)):
        first = max(0, c - (window - 1 if n else window))
        out["indices"] += [int(table[r, col]) for col in range(first // page_size, -(-(c + n) // page_size))]
        out["indptr"].append(len(out["indices"]))
        out["first_page_offset"].append(first % page_size if c + n else 0)
        for i in range(n if mask_words else 0):
            line = ancestors(parents[r] if parents is not None else None, i)[:window]
            out["tree_mask"].append(words_of(sum(1 << j for j in line), mask_words))
    return out


def rope_ref(x, weight, eps, positions, inv_freq, interleaved):
    """Norm (when weight is given) and rotation of x [T, H, D] in f64; returns (result, magnitude), the
    magnitude |x| + |partner| before the rotation, which bounds what f32 arithmetic can lose."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    out, mag = x.clone(), x.abs()
    half = len(inv_freq)
    for t in range(x.shape[0]):
        for j in range(half):
            a = float(positions[t]) * float(inv_freq[j])
            a0, b0 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            u, w = x[t, :, a0], x[t, :, b0]
            out[t, :, a0] = u * math.cos(a) - w * math.sin(a)
            out[t, :, b0] = w * math.cos(a) + u * math.sin(a)
            mag[t, :, a0] = mag[t, :, b0] = u.abs() + w.abs()
    return out, mag


def rope_tolerance(ref, mag, dtype):
    """One rounding to dtype, and 2^-19 of the magnitude: the mean square's sum (at most 2^-20 relative over 128
    terms added as a tree), the reciprocal root and three products (2^-22), the f32 angle (2^-23 radians) and its
    sine and cosine (2^-22)."""
    return ref.abs() * (torch.finfo(dtype).eps / 2) + mag * 2.0 ** -19


def attention_ref(q, k_pool, v_pool, indices, indptr, lpl, fpo, qo_indptr, scale, mask=None, qlen_rows=None):
    """out, lse2 [T, Hq, ...] in f64 of every query token over the keys it sees (keys behind a cleared bit are
    never touched), and the tolerances of both: (out, lse2, out_tol, lse_tol)."""
    T, hq, D = q.shape
    ps, hkv = k_pool.shape[1], k_pool.shape[2]
    G = hq // hkv
    eps = torch.finfo(q.dtype).eps
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    kf, vf = k_pool.flatten(0, 1), v_pool.flatten(0, 1)
    for r in range(len(lpl)):
        t0, t1 = int(qo_indptr[r]), int(qo_indptr[r + 1])
        n = t1 - t0
        ids = indices[int(indptr[r]):int(indptr[r + 1])].long()
        if n == 0 or len(ids) == 0:
            continue
        last = (len(ids) - 1) * ps + int(lpl[r])
        rows = (ids[:, None] * ps + torch.arange(ps)).reshape(-1)[int(fpo[r]):last]
        L = len(rows)
        for i in range(n):
            if mask is None:
                sees = list(range(i + 1))
            else:
                sees = [j for j in range(n) if (int(mask[t0 + i, j // 32]) >> (j % 32)) & 1]
            at = torch.cat((rows[:L - n], rows[L - n + torch.tensor(sees, dtype=torch.long)]))
            if len(at) == 0:
                continue
            k, v = kf[at].double(), vf[at].double()                       # [keys, hkv, D]
            qg = q[t0 + i].double().reshape(hkv, G, D)
            s = torch.einsum("hgd,khd->hgk", qg, k) * scale
            big = torch.einsum("hgd,khd->hgk", qg.abs(), k.abs()).amax(-1) * scale * LOG2E
            norm = torch.logsumexp(s, -1)
            p = torch.exp(s - norm[..., None])
            o = torch.einsum("hgk,khd->hgd", p, v)
            mean_abs = torch.einsum("hgk,khd->hgd", p, v.abs())
            out[t0 + i] = o.reshape(hq, D)
            lse[t0 + i] = (norm * LOG2E).reshape(hq)
            # a score's f32 sum of up to 128 products is off by at most 2^-17 of the sum of their sizes, in log2
            # units; exp2 and log2 add 2^-20.  P is rounded once to the type, the result once more.
            ds = big * 2.0 ** -17 + 2.0 ** -20
            tol_l[t0 + i] = (ds + 2.0 ** -20 * norm.abs()).reshape(hq)
            rel = eps / 2 + 2 * math.log(2.0) * ds + 2.0 ** -18
            tol_o[t0 + i] = (o.abs() * (eps / 2) + rel[..., None] * mean_abs).reshape(hq, D)
    return out, lse, tol_o, tol_l


def rows_attention_ref(q, k_pool, v_pool, seen, scale):
    """attention_ref of every query token alone, over the pool rows seen[t] (its own the last)."""
    one = lambda x: x.reshape(-1, 1, *x.shape[2:])
    parts = [attention_ref(q[t:t + 1], one(k_pool), one(v_pool), torch.tensor(rows), [0, len(rows)], [1], [0], [0, 1], scale)
             for t, rows in enumerate(seen)]
    return tuple(torch.cat(x) for x in zip(*parts))
