"""Rotary positions and the 4-bit cache: [summary] section 5's packed rows, each
turned by its own position before it attends, keys and values held in few bits.

Readings (the pages' models rotate queries and keys; none gives the formula):
  * a pair (x0, x1) of a head at position t is turned by t f_j radians as a
    point of the plane, pairs (j, j + rot / 2) or (2 j, 2 j + 1) of the first
    rot values;
  * MXFP4 (Open Compute Project, "Microscaling Formats"): e2m1 values, 32 of them
    with one power of two, which is the least whose 7 is no less than the
    largest of them.
Loops and tables in extended precision.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def rope(x, pos, freq, interleaved=False, factor=1.0):
    """x [n_rows][heads][d] turned by pos [n_rows]: float64 (rows of negative positions are NaN)."""
    y = np.array(x, dtype=np.longdouble)
    n = len(freq)
    for i, t in enumerate(pos):
        if t < 0:
            y[i] = np.nan
            continue
        for j in range(n):
            a = np.longdouble(int(t)) * np.longdouble(freq[j])
            c, s = factor * np.cos(a), factor * np.sin(a)
            u, v = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
            x0, x1 = np.longdouble(x[i, :, u]), np.longdouble(x[i, :, v])
            y[i, :, u], y[i, :, v] = x0 * c - x1 * s, x0 * s + x1 * c
    return y.astype(np.float64)


def mxfp4_power(block):
    """Exponent e of a block's power of two (its byte is e + 127)."""
    top = max(abs(float(v)) for v in block)
    if top == 0:
        return 0
    if math.isinf(top):
        return 125
    e = -120
    while e < 125 and top > 7.0 * 2.0 ** e:
        e += 1
    return e


def to_mxfp4(x):
    """(codes, bytes) of x [..., d]: codes 0 .. 15 [..., d], bytes [..., d / 32]."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, 32)
    codes, power = np.zeros(flat.shape, dtype=np.uint8), np.zeros(len(flat), dtype=np.uint8)
    levels = np.array(E2M1)
    for b, block in enumerate(flat):
        if np.isnan(block).any():
            power[b] = 255
            continue
        e = mxfp4_power(block)
        power[b] = e + 127
        a = np.minimum(np.abs(block) * 2.0 ** -e, 6.0)
        gap = np.abs(levels[None] - a[:, None])
        best = gap == gap.min(1, keepdims=True)
        # of two that are as near the even code
        even = best & (np.arange(8) % 2 == 0)[None]
        pick = np.where(even.any(1), even.argmax(1), best.argmax(1))
        codes[b] = pick + 8 * np.signbit(block)
    return codes.reshape(x.shape), power.reshape(*x.shape[:-1], -1)


def from_mxfp4(codes, power):
    """Values of codes [..., d] with bytes [..., d / 32] (255: NaN)."""
    levels = np.array(E2M1 + tuple(-v for v in E2M1))
    p = np.where(power == 255, np.nan, 2.0 ** (power.astype(np.float64) - 127))
    return levels[codes] * np.repeat(p, 32, axis=-1)
