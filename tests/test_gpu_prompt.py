"""Whole prompts on the GPU against the fp64 oracle, within derived bounds."""
import numpy as np
import pytest

import prompt_helpers as ph
from oracle import prompt as op

pytestmark = pytest.mark.gpu


def _i32(a, device="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)


def _check(got, want, D, dtype, rows=slice(None)):
    out, lse = (t.double().cpu().numpy() for t in got)
    tol_out, tol_lse = ph.attention_bounds(*want, D, dtype)
    assert np.isfinite(out[rows]).all()
    assert (np.abs(out - want[0]) <= tol_out)[rows].all(), np.max((np.abs(out - want[0]) / tol_out)[rows])
    fin = np.isfinite(want[1])
    np.testing.assert_array_equal(np.isneginf(lse)[rows], np.isneginf(want[1])[rows])
    err = np.where(fin, np.abs(np.where(fin, lse, 0.0) - np.where(fin, want[1], 0.0)), 0.0)
    assert (err <= tol_lse)[rows].all(), np.max((err - tol_lse)[rows])


ATTENTION = [  # dtype, D, H, G, lens, padding before, behind
    ("bf16", 128, 2, 4, [1], 0, 0),
    ("bf16", 128, 1, 1, [0, 2, 0], 0, 0),
    ("bf16", 128, 2, 4, [31, 32, 33, 0, 1, 64, 65, 129], 3, 5),
    ("bf16", 128, 1, 3, [200, 7], 0, 1),
    ("bf16", 64, 3, 2, [63, 64, 65, 130], 0, 0),
    ("bf16", 64, 1, 7, [5, 100], 2, 0),
    ("bf16", 96, 2, 5, [47, 1, 96], 0, 300),
    ("bf16", 96, 1, 1, [260], 0, 0),
    ("bf16", 256, 2, 8, [33, 40, 1], 1, 1),
    ("bf16", 256, 1, 1, [150, 129], 0, 0),
    ("bf16", 128, 1, 40, [9, 5], 0, 0),
    ("f32", 64, 2, 1, [1, 31, 32, 33, 100], 0, 0),
    ("f32", 64, 1, 4, [65, 0, 40], 4, 4),
    ("f32", 96, 2, 3, [50, 1], 0, 2),
    ("f32", 128, 1, 8, [33, 20], 0, 0),
    ("f32", 128, 2, 1, [140], 0, 0),
    ("f32", 256, 1, 2, [70, 1], 0, 1),
    ("f32", 256, 2, 4, [9], 0, 0),
]


@pytest.mark.parametrize("dtype,D,H,G,lens,before,behind", ATTENTION)
def test_attention(gpu_lib, dtype, D, H, G, lens, before, behind):
    rng = np.random.default_rng(D + G + len(lens))
    starts = before + np.concatenate([[0], np.cumsum(lens)])
    T = int(starts[-1]) + behind
    (q, k, v), host = ph.inputs(rng, T, H * G, H, D, dtype)
    got = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    _check(got, op.attention(*host, starts, D ** -0.5), D, dtype)


@pytest.mark.parametrize("dtype,scale", [("bf16", -0.2), ("bf16", 0.0), ("f32", -0.05), ("bf16", 3.0), ("f32", 1.0)])
def test_scales_and_contiguous_rows(gpu_lib, dtype, scale):
    """Negative scales, 0, and ones that leave a row with next to one weight."""
    rng = np.random.default_rng(5)
    starts, D = np.array([0, 90, 131]), 128
    (q, k, v), host = ph.inputs(rng, 131, 4, 2, D, dtype, fused=False)
    got = gpu_lib.prompt_attention(q, k, v, _i32(starts), scale=scale, return_lse=True)
    _check(got, op.attention(*host, starts, scale), D, dtype)


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("bf16", 64, 1), ("f32", 96, 2), ("bf16", 256, 3), ("f32", 256, 1),
                                       ("bf16", 96, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_memory_reaches_nothing(gpu_lib, dtype, D, G, bad):
    """What later tokens, other sequences and padding hold does not reach a
    query: their keys and values are not finite here."""
    rng = np.random.default_rng(8)
    starts, T = np.array([4, 74, 110, 110, 115]), 120
    (q, k, v), host = ph.inputs(rng, T, 2 * G, 2, D, dtype)
    hot = [40, 73, 100, 114]  # tokens whose own rows, and those behind them, do see it
    for t in (k, v):
        for i in (0, 1, 2, 3, 115, 119, *hot):
            t[i] = bad
    got = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    rows = np.ones(T, bool)
    for i in hot:
        first, last = next(r for r in op.ranges(starts, T) if r[0] <= i < r[1])
        rows[i:last] = False
    _check(got, op.attention(*host, starts, D ** -0.5), D, dtype, rows)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64), ("f32", 256)])
def test_infinite_values_are_added_where_they_are_seen(gpu_lib, dtype, D):
    """A single infinite value makes its channel infinite for the queries that
    see it, and changes no other channel and no other query."""
    rng = np.random.default_rng(9)
    starts, T, H, G = np.array([0, 50]), 50, 1, 2
    (q, k, v), host = ph.inputs(rng, T, H * G, H, D, dtype)
    clean = gpu_lib.prompt_attention(q, k, v, _i32(starts))
    v[20, 0, 7], v[33, 0, D - 1] = float("inf"), float("-inf")
    got = gpu_lib.prompt_attention(q, k, v, _i32(starts))
    want = clean.clone()
    want[20:, :, 7], want[33:, :, D - 1] = float("inf"), float("-inf")
    import torch
    assert torch.equal(got, want)


def test_extreme_scores(gpu_lib):
    """Rows whose scores are hugely negative, equal, or grow along the row."""
    import torch
    rng = np.random.default_rng(10)
    T, D = 150, 64
    (q, k, v), host = ph.inputs(rng, T, 2, 1, D, "f32")
    k.mul_(torch.linspace(-3.0, 3.0, T, device="cuda")[:, None, None])
    q[:40] *= 1e4
    k[60:90] = k[60].clone()
    host = [t.double().cpu().numpy() for t in (q, k, v)]
    got = gpu_lib.prompt_attention(q, k, v, _i32([0, T]), return_lse=True)
    _check(got, op.attention(*host, [0, T], D ** -0.5), D, "f32")


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 256), ("f32", 96)])
def test_the_largest_values_do_not_overflow(gpu_lib, dtype, D):
    """Values up to 2^100 under scores that grow by little along the row, so
    that weights stand above the held maximum."""
    import torch
    rng = np.random.default_rng(D)
    T = 700
    (q, k, v), _ = ph.inputs(rng, T, 2, 1, D, dtype)
    q.fill_(0.5)
    k.copy_(torch.linspace(0.0, 60.0 / D, T, device="cuda")[:, None, None])  # scores up to 30 * scale = 4 and below
    v.clamp_(-1.0, 1.0).mul_(2.0 ** 100 * (1 - 2.0 ** -7))
    host = [t.double().cpu().numpy() for t in (q, k, v)]
    for scale in (0.13, 1.1):
        got = gpu_lib.prompt_attention(q, k, v, _i32([0, T]), scale=scale, return_lse=True)
        _check(got, op.attention(*host, [0, T], scale), D, dtype)


def test_ranges_that_do_not_ascend_stay_inside(gpu_lib):
    """Whatever starts holds, rows are read and written inside [0, T) only, and
    a sequence that no other overlaps is right."""
    import torch
    rng = np.random.default_rng(11)
    T, D = 60, 64
    (q, k, v), host = ph.inputs(rng, T, 2, 1, D, "bf16")
    for starts in ([-5, 20, 70], [30, 10, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1], [60, 60], [0, 0, 0, 60]):
        got = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
        torch.cuda.synchronize()
        _check(got, op.attention(*host, starts, D ** -0.5), D, "bf16")


@pytest.mark.parametrize("dtype,G", [("bf16", 4), ("f32", 1)])
def test_clearing_leaves_the_rows_that_sequences_hold(gpu_lib, dtype, G):
    """Starts that descend, over more blocks than the card takes at once, so that
    the rows of no sequence are cleared when the others are long done: the same
    bits as with starts that ascend."""
    import torch
    rng = np.random.default_rng(16)
    T, H, D = 4000, 32, 64
    (q, k, v), _ = ph.inputs(rng, T, H * G, H, D, dtype)
    for starts, ascending in (([2000, 0, T], [0, 0, T]), ([3900, 0, 1700], [0, 1700, 1700])):
        out, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
        want = gpu_lib.prompt_attention(q, k, v, _i32(ascending), return_lse=True)
        held = max(ascending)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.isfinite(lse[:held]).all() and torch.isneginf(lse[held:]).all() and not out[held:].any()
    # out of order, none shares a row: rows behind the last are cleared, those between are anyone's
    got = gpu_lib.prompt_attention(q, k, v, _i32([2000, 3000, 100, 1500]), return_lse=True)
    want = gpu_lib.prompt_attention(q, k, v, _i32([100, 1500, 2000, 3000]), return_lse=True)
    for a, b in zip(got, want):
        for rows in (slice(0, 1500), slice(2000, T)):
            assert torch.equal(a[rows], b[rows])


def test_many_sequences(gpu_lib):
    """More sequences than a workgroup has threads, most of one token or none."""
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 3, 700)
    lens[300], lens[699] = 40, 33
    starts = np.concatenate([[0], np.cumsum(lens)])
    (q, k, v), host = ph.inputs(rng, int(starts[-1]) + 2, 2, 1, 64, "bf16")
    got = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    _check(got, op.attention(*host, starts, 0.125), 64, "bf16")


def test_blocks_of_few_sequences_in_any_order(gpu_lib):
    """Up to 64 sequences, whose blocks are handed out longest first: each block
    once, whatever the lengths."""
    rng = np.random.default_rng(15)
    for lens in ([0] * 63 + [90], [33] * 64, [0, 300, 0, 31, 32, 299, 1], list(rng.integers(0, 200, 64))):
        starts = 1 + np.concatenate([[0], np.cumsum(lens)])
        T = int(starts[-1]) + 40
        (q, k, v), _ = ph.inputs(rng, T, 4, 1, 64, "bf16")
        out, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
        more = _i32(np.concatenate([starts, [starts[-1]] * 70]))  # more than 64: the other way
        same = gpu_lib.prompt_attention(q, k, v, more, return_lse=True)
        import torch
        assert torch.equal(out, same[0]) and torch.equal(lse, same[1])
        assert (out[:1] == 0).all() and (out[starts[-1]:] == 0).all() and torch.isfinite(lse[1:starts[-1]]).all()
        for b in (0, len(lens) // 2, len(lens) - 1):
            first, last = int(starts[b]), int(starts[b + 1])
            if first < last:
                _check((out[first:last], lse[first:last]), _exact(q[first:last], k[first:last], v[first:last], 0.125), 64, "bf16")


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 64), ("bf16", 256)])
def test_many_blocks_in_order(gpu_lib, dtype, D):
    """64 ragged sequences, some empty, of more blocks than the card takes at
    once: these are handed out in order.  Each block once, the same bits as with
    more sequences, whose blocks are found another way."""
    import torch
    rng = np.random.default_rng(17)
    lens = rng.integers(0, 400, 64)
    lens[[0, 20, 21, 63]] = 0
    starts = 1 + np.concatenate([[0], np.cumsum(lens)])
    T, H = int(starts[-1]) + 2, 32
    assert (-(-T // 128) + 64) * H >= 4096
    (q, k, v), _ = ph.inputs(rng, T, H, H, D, dtype)
    got = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    more = gpu_lib.prompt_attention(q, k, v, _i32(np.concatenate([starts, [starts[-1]] * 9])), return_lse=True)
    assert torch.equal(got[0], more[0]) and torch.equal(got[1], more[1])
    assert torch.isneginf(got[1][:1]).all() and torch.isneginf(got[1][starts[-1]:]).all()
    for b in (1, 40, 62):
        rows = slice(starts[b], starts[b + 1])
        _check([t[rows] for t in got], _exact(q[rows], k[rows], v[rows], D ** -0.5), D, dtype)


def _exact(q, k, v, scale):
    """One sequence in 64 bits on the device: what op.attention gives."""
    import torch
    q, k, v = q.double(), k.double(), v.double()
    n, G = q.shape[0], q.shape[1] // k.shape[1]
    res = [[], [], [], []]
    for hq in range(q.shape[1]):
        kk, vv = k[:, hq // G].contiguous(), v[:, hq // G].contiguous()
        seen = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
        s = (scale * (q[:, hq].contiguous() @ kk.t().contiguous())).masked_fill(~seen, -torch.inf)
        p = torch.softmax(s, 1)
        big = (abs(scale) * (q[:, hq].abs().contiguous() @ kk.abs().t().contiguous())).masked_fill(~seen, 0.0).amax(1)
        for a, x in zip(res, (p @ vv, torch.logsumexp(s, 1), p @ vv.abs(), big)):
            a.append(x)
    out, lse, mag, big = (torch.stack(a, 1).cpu().numpy() for a in res)
    return out, lse, mag, big, np.broadcast_to(np.arange(1, n + 1)[:, None], lse.shape)


@pytest.mark.parametrize("dtype,D,H,G,n", [("bf16", 128, 2, 4, 2500), ("bf16", 256, 1, 8, 1111), ("f32", 64, 1, 2, 1501),
                                           ("bf16", 64, 1, 16, 3001), ("bf16", 96, 2, 1, 2047)])
def test_long_prompts(gpu_lib, dtype, D, H, G, n):
    rng = np.random.default_rng(n)
    (q, k, v), _ = ph.inputs(rng, n + 300, H * G, H, D, dtype)
    got = gpu_lib.prompt_attention(q, k, v, _i32([0, 300, n + 300]), return_lse=True)
    for first, last in ((0, 300), (300, n + 300)):
        _check([t[first:last] for t in got], _exact(q[first:last], k[first:last], v[first:last], D ** -0.5), D, dtype)


def test_the_same_call_gives_the_same_bits(gpu_lib):
    import torch
    rng = np.random.default_rng(13)
    (q, k, v), _ = ph.inputs(rng, 1000, 8, 2, 128, "bf16")
    starts = _i32([0, 1, 400, 1000])
    first = gpu_lib.prompt_attention(q, k, v, starts, return_lse=True)
    for _ in range(3):
        again = gpu_lib.prompt_attention(q, k, v, starts, return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    # a sequence's rows do not depend on what is packed beside it
    alone = gpu_lib.prompt_attention(q[400:], k[400:], v[400:], _i32([0, 600]), return_lse=True)
    assert all(torch.equal(a[400:], b) for a, b in zip(first, alone))


def test_empty_call_and_streams(gpu_lib):
    import torch
    rng = np.random.default_rng(14)
    (q, k, v), _ = ph.inputs(rng, 300, 8, 2, 128, "bf16")
    starts = _i32([0, 120, 300])
    out, lse = gpu_lib.prompt_attention(q[:0], k[:0], v[:0], starts, return_lse=True)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    want = gpu_lib.prompt_attention(q, k, v, starts)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gpu_lib.prompt_attention(q, k, v, starts)
    side.synchronize()
    assert torch.equal(got, want)
