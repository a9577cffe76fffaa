"""The packed verify batch over a paged key-value cache: places, cache values, attention.

[summary] section 5 (every request's rows to verify are laid end to end, and a
marker says which request and position a row belongs to); [blog]
"硬件感知前缀调度器" (K_b drafts of request b are verified, with the anchor
K_b + 1 rows).  Plain loops over requests, rows and pages; the attention in
float64 over the decoded values.

Readings:
  * the anchor and the drafts of a step are tokens len .. len + K of their
    request; len tokens are cached already, and accept_len drafts and the
    anchor stay (the emitted token is the next step's anchor);
  * free pages are a stack; requests pop and push in their own order.
"""
from __future__ import annotations

import math

import numpy as np


def pages_reserve(K, length, table, held, free_list, n_free, page_size, n_rows):
    """(t_offsets, row_req, row_pos, row_slot, table, held, n_free), or None
    where the batch does not fit."""
    table, held = np.array(table), np.array(held)
    top, offs, rows = int(n_free), [0], []
    for b in range(len(K)):
        if K[b] < -1 or length[b] < 0 or not 0 <= held[b] <= table.shape[1] or held[b] * page_size < length[b]:
            return None
        while held[b] * page_size < length[b] + K[b] + 1:
            if top == 0 or held[b] == table.shape[1]:
                return None
            top -= 1
            table[b, held[b]] = free_list[top]
            held[b] += 1
        for p in range(length[b], length[b] + K[b] + 1):
            rows.append((b, p, int(table[b, p // page_size]) * page_size + p % page_size))
        offs.append(len(rows))
    if len(rows) > n_rows:
        return None
    rows += [(-1, -1, -1)] * (n_rows - len(rows))
    req, pos, slot = np.array(rows, dtype=np.int64).reshape(-1, 3).T
    return np.array(offs), req, pos, slot, table, held, top


def pages_commit(length, accept_len, table, held, free_list, n_free, page_size, finished=None, n_pages=None):
    """(length, held, free_list, n_free), or None where an argument is invalid (page ids too, where n_pages is given)."""
    length, held, free = np.array(length), np.array(held), list(free_list)
    top = int(n_free)
    for b in range(len(length)):
        if accept_len[b] < -1 or length[b] < 0 or not 0 <= held[b] <= len(table[b]):
            return None
        length[b] = 0 if finished is not None and finished[b] else length[b] + accept_len[b] + 1
        keep = math.ceil(length[b] / page_size)
        if keep > held[b]:
            return None
        for p in range(keep, held[b]):
            if top == len(free) or n_pages is not None and not 0 <= table[b][p] < n_pages:
                return None
            free[top] = table[b][p]
            top += 1
        held[b] = keep
    return length, held, np.array(free), top


def e4m3_levels():
    """The non-negative e4m3 values in the order of their codes 0 .. 126: 4 bits of
    exponent (bias 7), 3 of mantissa, subnormal where the exponent is 0."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append((8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9)
    return np.array(out)


def to_e4m3(x):
    """The e4m3 value nearest each float64 (ties to the even code, magnitudes kept at 448)."""
    levels = e4m3_levels()
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(levels, np.where(np.isnan(a), 0, a)), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = levels[hi] - a, a - levels[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(x), np.nan, np.copysign(levels[code], x))


def attend(q, kcache, vcache, table, length, K, t_offsets, *, causal=True, scale, k_scale=None, v_scale=None):
    """(out, lse) of every packed row: softmax of scale * q . k over the keys
    the row sees, times the values.

    q [n_rows][Hq][D]; caches [n_pages][page][H][D]; query head h reads cache
    head h // (Hq / H).  Row i of request b sees tokens 0 .. length + i
    (causal) or 0 .. length + K.  Rows of no request are NaN."""
    n_rows, Hq, D = q.shape
    page, H = kcache.shape[1:3]
    group = Hq // H
    out = np.full((n_rows, Hq, D), np.nan)
    lse = np.full((n_rows, Hq), np.nan)
    for b in range(len(K)):
        for i in range(K[b] + 1):
            n = length[b] + (i if causal else K[b]) + 1
            t = np.arange(n)
            at = (np.asarray(table[b])[t // page], t % page)
            for h in range(Hq):
                k = kcache[at][:, h // group] * (1.0 if k_scale is None else float(k_scale[h // group]))
                v = vcache[at][:, h // group] * (1.0 if v_scale is None else float(v_scale[h // group]))
                s = scale * (k @ q[t_offsets[b] + i, h])
                with np.errstate(invalid="ignore"):
                    e = np.exp(s - s.max())
                    out[t_offsets[b] + i, h] = (e[:, None] * v).sum(0) / e.sum()
                    lse[t_offsets[b] + i, h] = s.max() + math.log(e.sum())
    return out, lse
