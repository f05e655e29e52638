"""fp64 oracle of the 8-bit paged cache: append, read back, attention.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product path.

A cache is a dict of numpy arrays: k_pages [pages, H, P, D] and v_pages
[pages, H, D, P] uint8 codes, k_scales and v_scales [pages, H] float32, and
"fmt", "e4m3" or "int8".
"""
from __future__ import annotations

import numpy as np

from .tree import tree_mask

QMAX = {"e4m3": 448.0, "int8": 127.0}


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 codes to fp64 values, from the formats' definitions."""
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    sign = np.where(codes >= 128, -1.0, 1.0)
    exp, mant = (codes >> 3) & 15, (codes & 7).astype(np.float64)
    mag = np.where(exp == 0, mant * 2.0 ** -9, (8.0 + mant) * np.exp2(exp.astype(np.float64) - 10.0))
    return sign * np.where((codes & 127) == 127, np.nan, mag)


def _e4m3_table():
    codes = np.arange(128, dtype=np.uint8)
    return decode(codes[:127], "e4m3")  # ascending magnitudes, code = index


def encode(y: np.ndarray, fmt: str) -> np.ndarray:
    """fp64 values in units of the scale to codes: nearest, ties to the even
    code; infinities saturate, NaN is 0x7f in e4m3 and 0 in int8."""
    y = np.asarray(y, dtype=np.float64)
    nan = np.isnan(y)
    c = np.clip(np.where(nan, 0.0, y), -QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return np.rint(c).astype(np.int8).view(np.uint8)
    tab = _e4m3_table()
    a = np.abs(c)
    hi = np.clip(np.searchsorted(tab, a), 1, 126)  # tab[hi-1] <= a <= tab[hi]
    lo = hi - 1
    dl, dh = a - tab[lo], tab[hi] - a
    idx = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))).astype(np.uint8)
    code = np.where(np.signbit(c), idx | 128, idx).astype(np.uint8)
    return np.where(nan, np.uint8(127), code)


def block_scale(values: np.ndarray, fmt: str) -> float:
    """The smallest power of two s >= 2^-126 with every finite |value| <= max * s."""
    v = np.abs(values[np.isfinite(values)])
    top = float(v.max()) if v.size else 0.0
    k = -126
    while top > QMAX[fmt] * 2.0 ** k:
        k += 1
    return 2.0 ** k


def _page(cache, table, b, col):
    if col >= table.shape[1]:
        return -1
    i = int(table[b, col])
    return i if 0 <= i < cache["k_pages"].shape[0] else -1


def append(cache, table, k, v, lengths, counts=None, index=None) -> np.ndarray:
    """In place; k, v [B, N, H, D] fp64 values.  Returns the new lengths."""
    B, N, H, D = k.shape
    P, fmt = cache["k_pages"].shape[2], cache["fmt"]
    out = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n0 = int(np.clip(lengths[b], 0, table.shape[1] * P))
        toks = list(range(N)) if index is None else [int(i) for i in index[b]]
        if counts is not None:
            toks = toks[: int(np.clip(counts[b], 0, N))]
        for i, t in enumerate(toks):
            if not 0 <= t < N or _page(cache, table, b, (n0 + i) // P) < 0:
                toks = toks[:i]
                break
        out[b] = n0 + len(toks)
        pos = n0
        while pos < out[b]:
            col = pos // P
            page = _page(cache, table, b, col)
            t0, t1 = pos - col * P, min(int(out[b]) - col * P, P)
            src = toks[pos - n0: pos - n0 + t1 - t0]
            for h in range(H):
                for name, x in (("k", k), ("v", v)):
                    codes = cache[name + "_pages"][page, h]
                    codes = codes if name == "k" else codes.T  # [P, D]
                    new = x[b, src, h]
                    s_old, s = float(cache[name + "_scales"][page, h]), block_scale(new, fmt)
                    if t0 > 0:
                        s = max(s, s_old)
                        if s > s_old:
                            codes[:t0] = encode(decode(codes[:t0], fmt) * (s_old / s), fmt)
                    codes[t0:t1] = encode(new / s, fmt)
                    cache[name + "_scales"][page, h] = s
            pos = col * P + t1
    return out


def values(cache, table, b, n):
    """Positions 0..n-1 of sequence b: k, v [n, H, D] fp64, seen [n] (False without a page)."""
    P, H, D = cache["k_pages"].shape[2], cache["k_pages"].shape[1], cache["k_pages"].shape[3]
    k, v, seen = np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros(n, dtype=bool)
    for c0 in range(0, n, P):
        page = _page(cache, table, b, c0 // P)
        if page < 0:
            continue
        m = min(P, n - c0)
        seen[c0:c0 + m] = True
        k[c0:c0 + m] = (decode(cache["k_pages"][page, :, :m], cache["fmt"]) *
                        cache["k_scales"][page].astype(np.float64)[:, None, None]).transpose(1, 0, 2)
        v[c0:c0 + m] = (decode(cache["v_pages"][page, :, :, :m], cache["fmt"]) *
                        cache["v_scales"][page].astype(np.float64)[:, None, None]).transpose(2, 0, 1)
    return k, v, seen


def read(cache, table, lengths, T, starts=None):
    """k, v [B, T, H, D] fp64."""
    B = len(lengths)
    P, H, D = cache["k_pages"].shape[2], cache["k_pages"].shape[1], cache["k_pages"].shape[3]
    out = [np.zeros((B, T, H, D)) for _ in range(2)]
    for b in range(B):
        n = int(np.clip(lengths[b], 0, table.shape[1] * P))
        s = max(0, int(starts[b])) if starts is not None else 0
        m = min(T, n - s)
        if m > 0:
            k, v, _ = values(cache, table, b, s + m)
            out[0][b, :m], out[1][b, :m] = k[s:], v[s:]
    return out


def node_sets(parents, N):
    """see[i, j]: node i sees node j (itself and its ancestors; a node whose
    parent is not in [0, i) sees only itself); parents None: a chain."""
    if parents is None:
        return np.tril(np.ones((N, N), dtype=bool))
    return tree_mask(parents)[0].astype(bool)


def attention(cache, table, q, lengths, scale, k_new=None, v_new=None, parents=None, num_nodes=None):
    """q [B, N, Hq, D] fp64.  Returns out [B, N, Hq, D], lse [B, N, Hq], and
    what error bounds need: sum_j p_j |v_j| (out's shape), the largest
    scale * sum |q| |k_j| over what a query sees and the number it sees ([B, N, Hq])."""
    B, N, Hq, D = q.shape
    H, P = cache["k_pages"].shape[1], cache["k_pages"].shape[2]
    G = Hq // H
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, big, cnt = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    for b in range(B):
        n = int(np.clip(lengths[b], 0, table.shape[1] * P))
        k, v, seen = values(cache, table, b, n)
        see = node_sets(None if parents is None else parents[b], N)
        nn = N if num_nodes is None else int(np.clip(num_nodes[b], 0, N))
        for i in range(nn):
            for hq in range(Hq):
                h = hq // G
                kk, vv = k[seen, h], v[seen, h]
                if k_new is not None:
                    kk = np.concatenate([kk, k_new[b, see[i], h]])
                    vv = np.concatenate([vv, v_new[b, see[i], h]])
                if len(kk) == 0:
                    continue
                s = scale * (kk @ q[b, i, hq])
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                lse[b, i, hq] = m + np.log(z)
                out[b, i, hq] = (e / z) @ vv
                mag[b, i, hq] = (e / z) @ np.abs(vv)
                big[b, i, hq] = abs(scale) * (np.abs(kk) @ np.abs(q[b, i, hq])).max()
                cnt[b, i, hq] = len(kk)
    return out, lse, mag, big, cnt
