"""Penalties, biases and grammar masks on the logits of a request's rows.

[blog] "形式化定义": the target scores every drafted position of a request in one
pass, so row i follows the history and the first i drafts.  Plain loops over
the tokens, float64.
"""
from __future__ import annotations

import numpy as np

MASKED = float(np.float32(-1.0e30))    # the float that is written


def constrain(logits, *, prompt=(), written=(), drafts=(), rep=1.0, freq=0.0, pres=0.0, bias=(), allowed=None):
    """Rows [n][V] of one request: row i after ``prompt``, ``written`` and
    drafts[:i]; bias: (id, value) pairs; allowed: bool [n][V] or None."""
    out = np.array(logits, dtype=np.float64)
    n, V = out.shape
    for i in range(n):
        count = np.zeros(V)
        for t in list(written) + list(drafts[:i]):
            count[t] += 1
        seen = count > 0
        for t in prompt:
            seen[t] = True
        row = out[i]
        with np.errstate(invalid="ignore", over="ignore"):
            row[seen] = np.where(row[seen] > 0, row[seen] / rep, row[seen] * rep)
            row -= freq * count + pres * (count > 0)
        for t, x in bias:
            row[t] += x
        row[row < MASKED] = MASKED
        if allowed is not None:
            row[~np.asarray(allowed[i], dtype=bool)] = MASKED
    return out
