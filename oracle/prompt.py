"""fp64 oracle of whole prompts: causal attention of packed sequences.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product path.
"""
from __future__ import annotations

import numpy as np


def ranges(starts, T):
    """The token ranges of the sequences, clamped as the library does."""
    out = []
    for b in range(len(starts) - 1):
        first = int(np.clip(starts[b], 0, T))
        out.append((first, int(np.clip(starts[b + 1], first, T))))
    return out


def attention(q, k, v, starts, scale):
    """q [T, Hq, D], k and v [T, H, D] fp64.  Returns out [T, Hq, D], lse [T,
    Hq], and what error bounds need: sum_j p_j |v_j| (out's shape), the largest
    |scale| sum |q| |k_j| over what a query sees and the number it sees ([T, Hq])."""
    T, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, big, cnt = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    for first, last in ranges(starts, T):
        for i in range(first, last):
            for hq in range(Hq):
                kk, vv = k[first:i + 1, hq // G], v[first:i + 1, hq // G]
                s = scale * (kk @ q[i, hq])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                lse[i, hq] = m + np.log(z)
                out[i, hq] = (e / z) @ vv
                mag[i, hq] = (e / z) @ np.abs(vv)
                big[i, hq] = abs(scale) * (np.abs(kk) @ np.abs(q[i, hq])).max()
                cnt[i, hq] = i + 1 - first
    return out, lse, mag, big, cnt
