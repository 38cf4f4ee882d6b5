"""Attention over 8-bit pages in float64 with a bound that goes by what a row sees
and by what of it has weight, where ``tests/_paged.py`` has the largest value of
the sequence.

A weight times its page's scale is held in fp16, relative to a power of two that
is at most the row's largest such product (the power only follows that by steps,
upwards): it is off by 2^-11 of itself, or in fp16's subnormal range by 2^-25 of the power.
Stored values are at most 448. So with w_j the weights of a sum of 1 and s_j the
scales of the values' pages the last term is

  n 2^-25 448 max_j w_j s_j     in the place of   n 2^-25 max_j |v_j|.
"""
import numpy as np


def reference(b):
    """(o, bound) [tp, used, hq, d] of a ``tests._paged.Batch`` whose rows all lie within the pages."""
    lay, G = b.lay, b.lay.group
    o = np.zeros((lay.tp, b.used, lay.hq, lay.d))
    bound = np.zeros_like(o)
    for s, (n, c) in enumerate(zip(b.new, b.cached)):
        end = n + c
        if n == 0:
            continue
        hidden = np.arange(end)[None, :] > (c + np.arange(n))[:, None]
        ids = b.table[s, :-(-end // b.page)]
        for r in range(lay.tp):
            keys, vals = b.keys("k", s, r, end), b.keys("v", s, r, end)
            scale = np.repeat(b.scale["v"][r, ids].T, b.page, 1)[:, :end]
            for h in range(lay.hq):
                x = b.q[r, b.cu[s]:b.cu[s] + n, h]
                k, v = keys[h // G], vals[h // G]
                t = np.where(hidden, -np.inf, x @ k.T / np.sqrt(lay.d))
                w = np.exp(t - t.max(-1, keepdims=True))
                w = w / w.sum(-1, keepdims=True)
                mag = np.where(hidden, 0, np.abs(x) @ np.abs(k).T).max(-1) / np.sqrt(lay.d)
                low = 2.0 ** -17 * np.abs(x).max(-1) * np.where(hidden, 0, np.abs(k).sum(-1)).max(-1) / np.sqrt(lay.d)
                cc = 2 * (2 * lay.d + 4) * 2.0 ** -24 * mag + 2 * low + 2.0 ** -21 + 2 * end * 2.0 ** -24 + 2.0 ** -17
                oo, A = w @ v, w @ np.abs(v)
                small = end * 2.0 ** -25 * 448 * (w * scale[h // G]).max(-1, keepdims=True)
                rows = slice(b.cu[s], b.cu[s] + n)
                o[r, rows, h] = oo
                bound[r, rows, h] = (1 + 2.0 ** -6) * (2.0 ** -8 * np.abs(oo) + (2.0 ** -11 + cc[:, None]) * A + small)
    return o, bound
