"""The prompts' oracle against hand-made values and torch's own softmax (CPU)."""
import numpy as np
import torch

from oracle import prompt as op


def test_ranges_are_clamped():
    assert op.ranges([0, 3, 3, 9], 7) == [(0, 3), (3, 3), (3, 7)]
    assert op.ranges([-2, 5, 1, 4], 6) == [(0, 5), (5, 5), (1, 4)]


def test_one_token_and_none():
    q = np.ones((3, 2, 4))
    k = np.arange(12.0).reshape(3, 1, 4)
    out, lse, *_ = op.attention(q, k, k, [1, 2, 2], 0.5)
    assert (out[[0, 2]] == 0).all() and (lse[[0, 2]] == -np.inf).all()
    assert (out[1] == k[1]).all() and (lse[1] == 0.5 * k[1].sum()).all()


def test_is_torchs_softmax():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(9, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    out, lse, mag, big, cnt = op.attention(q, k, v, [0, 4, 9], -0.3)
    for first, last in ((0, 4), (4, 9)):
        for hq in range(4):
            s = torch.from_numpy(q[first:last, hq] @ k[first:last, hq // 2].T * -0.3)
            s = s.masked_fill(torch.ones_like(s).triu(1).bool(), -torch.inf)
            np.testing.assert_allclose(out[first:last, hq], torch.softmax(s, 1).numpy() @ v[first:last, hq // 2])
            np.testing.assert_allclose(lse[first:last, hq], torch.logsumexp(s, 1).numpy())
    assert (np.abs(out) <= mag + 1e-12).all() and cnt[8, 0] == 5
