"""The budget's oracle against hand-made values and its own conservation laws (CPU)."""
import numpy as np

import kv_helpers as kh
from oracle import budget as ob
from oracle import kv as okv
from oracle import prompt as op


def test_every_query_gives_a_weight_of_one():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(9, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    starts = [1, 5, 5, 9]
    _, lse, *_ = op.attention(q, k, v, starts, 0.4)
    w = ob.prompt_weights(q, k, lse, starts, 0.4, 6)[0]
    np.testing.assert_allclose(w.sum(2), [[8, 8], [0, 0], [8, 8]])
    assert (w[0, :, 4:] == 0).all()
    np.testing.assert_allclose(ob.prompt_weights(q, k, lse, starts, 0.4, 2)[0], w[:, :, :2])


def test_kept_nodes_give_theirs_to_cache_and_path():
    rng = np.random.default_rng(1)
    lens, P, H, D, N = [20, 0, 7], 16, 2, 64, 5
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D, extra=N)
    q, k, v = rng.normal(size=(3, N, 4, D)), rng.normal(size=(3, N, H, D)), rng.normal(size=(3, N, H, D))
    index = np.array([[0, 1, 2, 3, 4], [0, 2, -1, 0, 0], [-1, 0, 0, 0, 0]])
    # each kept node sees the cache and the path up to itself
    lse = np.full((3, N, 4), np.nan)
    for b in range(3):
        nodes = ob.kept_nodes(b, N, None, index)
        for i, n in enumerate(nodes):
            at = nodes[:i + 1]
            lse[b, n] = okv.attention(c, table[b:b + 1], q[b:b + 1, at], lens[b:b + 1], 0.1, k[b:b + 1, at],
                                      v[b:b + 1, at])[1][0, -1]
    old = rng.random((3, H, table.shape[1] * P)).astype(np.float32)
    got, written = ob.kv_weights(c, table, q, lse, lens, old, 0.1, k, None, index)
    assert written.sum(1).tolist() == [25, 2, 7]
    for b, n in enumerate((5, 2, 0)):
        added = got[0, b, :, :lens[b] + n].sum(1) - old[b, :, :lens[b]].astype(np.float64).sum(1)
        np.testing.assert_allclose(added, 2.0 * n)


def test_what_stays():
    w = np.array([3.0, 1.0, np.nan, 1.0, 0.0, 1.0, -0.0, 9.0], np.float32)
    assert ob.kept_positions(w, 8, 4, 1).tolist() == [0, 1, 3, 7]
    assert ob.kept_positions(w, 8, 7, 0).tolist() == [0, 1, 3, 4, 5, 6, 7]
    assert ob.kept_positions(w, 7, 3, 3).tolist() == [4, 5, 6]


def test_eviction_keeps_values():
    rng = np.random.default_rng(2)
    P, H, D, lens = 16, 2, 64, [40, 10]
    c, table = kh.make_cache(rng, "int8", lens, P, H, D, extra=60, spare=0, poison=False)
    w = rng.random((2, H, table.shape[1] * P)).astype(np.float32)
    before = [okv.values(c, table, b, lens[b])[:2] for b in range(2)]
    new = table[:, 4:6].copy()  # pages that hold nothing
    t2, l2, w2, kept = ob.evict(c, table, lens, w, new, 20, 5, 30)
    assert l2.tolist() == [20, 10] and (kept[1] == -1).all() and (t2[1] == table[1]).all()
    after = okv.values(c, t2, 0, 20)
    for h in range(H):
        assert (np.diff(kept[0, h]) > 0).all() and kept[0, h, 15:].tolist() == [35, 36, 37, 38, 39]
        np.testing.assert_array_equal(w2[0, h, :20], w[0, h, kept[0, h]])
        for x, y, name in zip(before[0], after[:2], "kv"):
            step = c[name + "_scales"][t2[0, :2], h].max()
            assert (np.abs(y[:, h] - x[kept[0, h], h]) <= step / 2).all()
