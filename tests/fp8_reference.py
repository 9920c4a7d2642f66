"""Plain 64-bit references of the 8-bit cache's operators for the tests: e4m3 codes and exponents of an append, and
which pool rows a token sees under a window with sinks.  They share nothing with the library.
"""
from __future__ import annotations

import math

import torch

import step_reference as R

E4M3 = torch.float8_e4m3fn
EXP_MIN, EXP_MAX = -15, 7


def code_of(y: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value of y (f64), ties to even, magnitudes above 448 to 448; as f64."""
    a = y.abs()
    e = torch.frexp(a)[1].double() - 1                        # 2^e <= a < 2^(e + 1)
    step = torch.exp2(torch.clamp(e, min=-6) - 3)
    return torch.clamp(torch.round(a / step) * step, max=448.0) * torch.sign(y)


def need_of(top: float) -> int:
    """The least exponent whose largest code holds top."""
    e = EXP_MIN
    while e < EXP_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def values(pool: torch.Tensor, exps: torch.Tensor) -> torch.Tensor:
    """What the cache holds, as f16 (exactly)."""
    e = exps.long().clamp(EXP_MIN, EXP_MAX).double()
    wide = pool.float().double() * torch.exp2(e)[:, None, :, None]
    assert torch.equal(wide.half().double().nan_to_num(7.0), wide.nan_to_num(7.0))
    return wide.half()


def append_ref(x, mag, pool, exps, slots, got=None):
    """x [T, Hkv, D] (f64, to be held) and mag (rope_ref's) into pool / exps (CPU): (lowest, highest) codes that a
    result may have, as f64, and its exponents.  f32 arithmetic knows x to 2^-19 of mag (rope_tolerance): where a run's
    maximum lies that close to a border between two exponents either is right, and the result's own (got) is taken."""
    P, ps, hkv, D = pool.shape
    low, exps = pool.float().double(), exps.long().clone()
    high = low.clone()
    rows = P * ps
    runs, before = [], -1
    for t, s in enumerate(slots.tolist()):
        page = s // ps if 0 <= s < rows else -1
        if page >= 0 and page == before:
            runs[-1][1].append(t)
        elif page >= 0:
            runs.append((page, [t]))
        before = page
    for page, toks in runs:
        at = torch.tensor([int(slots[t]) % ps for t in toks])
        first = int(at.min())
        for h in range(hkv):
            y = x[toks, h]
            fine = y.isfinite()
            top = float(y[fine].abs().max()) if fine.any() else 0.0
            sure = mag[toks, h][fine] * 2.0 ** -19
            most = float((y[fine].abs() + sure).max()) if fine.any() else 0.0
            least = float((y[fine].abs() - sure).max()) if fine.any() else 0.0
            e = need_of(top)
            if got is not None and need_of(least) != need_of(most):
                e = min(max(int(got[page, h]), need_of(least)), need_of(most))
            if first > 0:
                old = min(max(int(exps[page, h]), EXP_MIN), EXP_MAX)
                if old >= e:
                    e = old
                else:
                    for side in (low, high):
                        side[page, :first, h] = code_of(side[page, :first, h] * 2.0 ** (old - e))
            exps[page, h] = e
            tol = mag[toks, h] * 2.0 ** -19
            y = torch.where(fine, y, torch.nan)
            low[page, at, h], high[page, at, h] = code_of((y - tol) / 2.0 ** e), code_of((y + tol) / 2.0 ** e)
    return low, high, exps


def seen_rows(ids, page_size, first, length, new, i, window=0, sinks=0, line=None, depth=None):
    """Pool rows that new token i of a request sees: `length` listed rows from `first` on, the last `new` of them new.
    line: the new tokens that its mask shows (None: a chain); depth: how far behind the first new token it stands."""
    total, ds = first + length, first + length - new
    at = ds + (i if depth is None else depth)
    out = []
    for y in range(first, total):
        if y >= ds and line is not None:
            ok = (y - ds) in line
        else:
            ok = y <= (ds + i if line is None else ds - 1) and (window == 0 or y < sinks or y > at - window)
        if ok:
            out.append(int(ids[y // page_size]) * page_size + y % page_size)
    return out


def attention_ref(q, k_rows, v_rows, seen, scale):
    """rows_attention_ref, with zeros and -inf for a token that sees nothing."""
    empty = [not rows for rows in seen]
    out = R.rows_attention_ref(q, k_rows, v_rows, [rows or [0] for rows in seen], scale)
    for t, nothing in enumerate(empty):
        if nothing:
            out[0][t], out[1][t], out[2][t], out[3][t] = 0.0, -math.inf, 0.0, 0.0
    return out
