"""64-bit reference of the rotary positions (numpy), with an element-wise bound on how far a kernel
that works in fp32 and rounds its result once can be from it.

Bound of y = x cos t - z sin t: the angle, as a fraction of a turn with 24 significant bits, is off
by at most 2 pi 2^-25 < 2^-22 rad, cos and sin in fp32 by 2^-22 more together with the products and
the sum (three roundings of 2^-24 of at most |x| + |z|): 2^-20 (|x| + |z|) covers them.  The store
adds half a step, u |y| (fp16 below 2^-14: at most 2^-25)."""

import math

import numpy as np

from tests.cache_ref import SUB, U16


def turned(x, pos, freqs, axes, rotary, interleaved, dt, sign=1.0):
    """x [B, L, heads, D] turned, and the bound; pos [axes, B, L]."""
    x = np.asarray(x, dtype=np.float64)
    y, err = x.copy(), np.zeros_like(x)
    n = rotary // 2
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # whole positions: the product is exact in integers where a float would round
        turns = np.vectorize(lambda p: math.fmod(int(p) * freqs[i] / (2 * math.pi), 1.0) if abs(int(p)) < 2 ** 20
                             else float((int(p) * round(freqs[i] / (2 * math.pi) * 2 ** 80)) % 2 ** 80) / 2 ** 80,
                             otypes=[np.float64])(pos[axes[i]])
        c, s = (f(2 * math.pi * turns)[:, :, None] for f in (np.cos, np.sin))
        s = s * sign
        u, v = x[..., a], x[..., b]
        y[..., a], y[..., b] = u * c - v * s, u * s + v * c
        for d in (a, b):
            err[..., d] = 2.0 ** -20 * (np.abs(u) + np.abs(v)) + U16[dt] * np.abs(y[..., d]) + SUB[dt]
    return y, err
