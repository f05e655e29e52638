"""fp64 oracle of the cache under a budget: gathered attention weights and
eviction.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product path.
A cache is the dict of oracle/kv.py.
"""
from __future__ import annotations

import numpy as np

from . import kv as okv
from .prompt import ranges


def _gather(q, k, lse, scale, sees):
    """Weights [keys] of queries q [n, D] over keys k, and what error bounds
    need: sum e * |scale| sum |q||k|, sum e * (|lse| + |s|), queries that count."""
    s = scale * (q @ k.T)
    count = sees & ~np.isinf(lse)[:, None]  # e^-inf is 0, and a query that saw nothing counts for nothing
    at = np.where(np.isfinite(lse), lse, 0.0)
    e = np.where(count, np.exp(np.where(count, s - at[:, None], 0.0)), 0.0)
    big = abs(scale) * (np.abs(q) @ np.abs(k).T)
    return np.stack([e.sum(0), (e * big).sum(0), (e * (np.abs(at)[:, None] + np.abs(s))).sum(0), count.sum(0)])


def prompt_weights(q, k, lse, starts, scale, capacity):
    """[4, B, H, capacity]: the weights, and _gather's other sums."""
    T, Hq, _ = q.shape
    H = k.shape[1]
    out = np.zeros((4, len(starts) - 1, H, capacity))
    for b, (first, last) in enumerate(ranges(starts, T)):
        n = last - first
        m = min(n, capacity)
        for hq in range(Hq):
            got = _gather(q[first:last, hq], k[first:last, hq // (Hq // H)], lse[first:last, hq], scale,
                          np.tril(np.ones((n, n), bool)))
            out[:, b, hq // (Hq // H), :m] += got[:, :m]
    return out


def kept_nodes(b, N, counts, index):
    nodes = list(range(N)) if index is None else [int(i) for i in index[b]]
    if counts is not None:
        nodes = nodes[: int(np.clip(counts[b], 0, N))]
    for i, n in enumerate(nodes):
        if not 0 <= n < N:
            return nodes[:i]
    return nodes


def kv_weights(cache, table, q, lse, lengths, weights, scale, k_new=None, counts=None, index=None):
    """[4, B, H, capacity] as prompt_weights (the old weights added), and which
    positions are written."""
    B, N, Hq, _ = q.shape
    P, H = cache["k_pages"].shape[2], cache["k_pages"].shape[1]
    C = weights.shape[2]
    out, written = np.zeros((4, B, H, C)), np.zeros((B, C), bool)
    for b in range(B):
        n = int(np.clip(lengths[b], 0, table.shape[1] * P))
        nodes = kept_nodes(b, N, counts, index)
        k, _, seen = okv.values(cache, table, b, n)
        m = min(len(nodes) if k_new is not None else 0, C - n)
        written[b, :n + m] = True
        out[0, b, :, :n] = weights[b, :, :n]
        if not nodes:
            continue
        for hq in range(Hq):
            h = hq // (Hq // H)
            got = _gather(q[b, nodes, hq], k[:, h], lse[b, nodes, hq], scale, np.tile(seen, (len(nodes), 1)))
            out[:, b, h, :n] += np.where(seen, got, 0.0)
            if k_new is not None:
                got = _gather(q[b, nodes, hq], k_new[b, nodes, h], lse[b, nodes, hq], scale,
                              np.tril(np.ones((len(nodes), len(nodes)), bool)))
                out[:, b, h, n:n + m] += got[:, :m]
    return out, written


def kept_positions(w, n, budget, recent):
    """The positions of w[0..n) that stay: ties to the lowest, NaN below all."""
    key = np.where(np.isnan(w[:n - recent]), -np.inf, w[:n - recent])
    nan = np.isnan(w[:n - recent])
    order = sorted(range(n - recent), key=lambda i: (nan[i], -key[i], i))
    return np.array(sorted(order[:budget - recent]) + list(range(n - recent, n)), dtype=np.int64)


def evict(cache, table, lengths, weights, new_pages, budget, recent, limit):
    """In place on the cache; returns (table, lengths, weights, kept)."""
    B, H, C = weights.shape
    P, fmt, pages = cache["k_pages"].shape[2], cache["fmt"], cache["k_pages"].shape[0]
    out_table, out_len = table.copy(), np.zeros(B, np.int32)
    out_w, kept = np.zeros(weights.shape, np.float32), np.full((B, H, budget), -1, np.int32)
    old = {n: (x.copy() if isinstance(x, np.ndarray) else x) for n, x in cache.items()}
    for b in range(B):
        n = int(np.clip(lengths[b], 0, table.shape[1] * P))
        if n <= limit:
            out_len[b], out_w[b, :, :n] = n, weights[b, :, :n]
            continue
        out_len[b] = budget
        out_table[b] = -1
        out_table[b, :new_pages.shape[1]] = new_pages[b]
        for h in range(H):
            at = kept_positions(weights[b, h], n, budget, recent)
            kept[b, h], out_w[b, h, :budget] = at, weights[b, h, at]
            for d0 in range(0, budget, P):
                to = int(new_pages[b, d0 // P])
                if not 0 <= to < pages:
                    continue
                src = at[d0:d0 + P]
                for name in ("k", "v"):
                    codes, unit = np.zeros((len(src), cache["k_pages"].shape[3]), np.uint8), np.zeros(len(src))
                    for i, t in enumerate(src):
                        page = okv._page(cache, table, b, t // P)
                        if page >= 0:
                            blk = old[name + "_pages"][page, h]
                            codes[i] = blk[t % P] if name == "k" else blk[:, t % P]
                            unit[i] = old[name + "_scales"][page, h]
                    x = okv.decode(codes, fmt) * unit[:, None]
                    s = okv.block_scale(x, fmt)
                    code = okv.encode(x / s, fmt)
                    dst = cache[name + "_pages"][to, h]
                    (dst if name == "k" else dst.T)[:len(src)] = code
                    cache[name + "_scales"][to, h] = s
    return out_table, out_len, out_w, kept
