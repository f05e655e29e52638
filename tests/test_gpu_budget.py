"""The cache under a budget on the GPU against the fp64 oracle: gathered
weights within derived bounds, eviction bit for bit."""
import numpy as np
import pytest

import kv_helpers as kh
import prompt_helpers as ph
from oracle import budget as ob
from oracle import kv as okv
from oracle import prompt as op

pytestmark = pytest.mark.gpu

U = ph.U


def _i32(a, device="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)


def _f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _weights_close(got, want, D, rows=None):
    """Each weight e^(s - lse) is off by its score's error, by the rounding of
    s, of lse and of their difference in log2 (each 2 u of their magnitudes),
    by exp2's few u, and the sum over cnt terms by cnt u."""
    w, big, mag, cnt = want
    tol = 1.01 * (ph.score_error(big, D) + 4 * U * mag + (cnt + 8) * U * np.abs(w)) + 1e-37
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - w) <= tol)
    if rows is not None:
        bad &= rows
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], w[bad][:4], tol[bad][:4])


# ------------------------------------------------------------- prompts --
PROMPTS = [  # dtype, D, H, G, lens, capacity
    ("bf16", 128, 2, 4, [1], 1),
    ("bf16", 128, 1, 1, [0, 2, 0, 130], 200),
    ("bf16", 128, 2, 4, [31, 32, 33, 0, 1, 64, 65, 129], 129),
    ("bf16", 128, 1, 3, [260, 7], 300),
    ("bf16", 64, 3, 2, [63, 64, 65, 130], 70),
    ("bf16", 64, 1, 7, [5, 100], 1000),
    ("bf16", 96, 2, 5, [47, 1, 96], 96),
    ("bf16", 256, 2, 8, [33, 40, 1], 41),
    ("f32", 64, 2, 1, [1, 31, 32, 33, 100], 100),
    ("f32", 96, 2, 3, [50, 1], 64),
    ("f32", 128, 1, 8, [33, 140], 140),
    ("f32", 256, 1, 2, [70, 1], 70),
]


@pytest.mark.parametrize("dtype,D,H,G,lens,capacity", PROMPTS)
def test_prompt_weights(gpu_lib, dtype, D, H, G, lens, capacity):
    rng = np.random.default_rng(D + G + len(lens))
    starts = 2 + np.concatenate([[0], np.cumsum(lens)])
    T = int(starts[-1]) + 3
    (q, k, v), host = ph.inputs(rng, T, H * G, H, D, dtype)
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    got = gpu_lib.prompt_weights(q, k, lse, _i32(starts), capacity)
    _weights_close(got, ob.prompt_weights(*host[:2], lse.double().cpu().numpy(), starts, D ** -0.5, capacity), D)
    if capacity >= max(lens):  # every query of every head gives a weight of 1, but for two scores' errors: (6 D + 48) u
        np.testing.assert_allclose(got.sum(2).cpu().numpy(), np.outer(lens, [G] * H), rtol=2e-3)  # times at most 20 here


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 3), ("bf16", 64, 7), ("f32", 64, 5), ("bf16", 96, 33), ("bf16", 256, 12)])
def test_prompt_weights_of_groups_of_any_size(gpu_lib, dtype, D, G):
    """Groups that do not divide a tile's rows; queries before a key hold NaN,
    and the weights of the keys behind them are as they were."""
    rng = np.random.default_rng(G)
    n, H = 190, 1
    (q, k, v), host = ph.inputs(rng, n, H * G, H, D, dtype)
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32([0, n]), return_lse=True)
    want = ob.prompt_weights(*host[:2], lse.double().cpu().numpy(), [0, n], D ** -0.5, n)
    _weights_close(gpu_lib.prompt_weights(q, k, lse, _i32([0, n]), n), want, D)
    for bad in (0, 41, 127, 150):
        x = q.clone()
        x[bad] = float("nan")
        rows = np.broadcast_to(np.arange(n) > bad, want.shape[1:])
        _weights_close(gpu_lib.prompt_weights(x, k, lse, _i32([0, n]), n), want, D, rows)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_prompt_weights_of_statistics_that_are_not_finite(gpu_lib, dtype, D):
    """lse of -infinity and +infinity weighs nothing; what other sequences and
    padding hold reaches nothing, nor do the queries before a key."""
    rng = np.random.default_rng(3)
    starts, T = np.array([5, 75, 140]), 150
    (q, k, v), host = ph.inputs(rng, T, 4, 2, D, dtype)
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    lse[10:12], lse[80, 1] = -float("inf"), float("inf")
    lse[:5] = lse[140:] = float("nan")
    q[:5] = q[140:] = k[:5] = k[140:] = float("nan")
    q[5:9] = float("nan")       # the queries before key 4 of sequence 0
    want = ob.prompt_weights(*host[:2], lse.double().cpu().numpy(), starts, -0.1, 80)
    got = gpu_lib.prompt_weights(q, k, lse, _i32(starts), 80, scale=-0.1)
    rows = np.ones(got.shape, bool)
    rows[0, :, :4] = False
    _weights_close(got, want, D, rows)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("bf16", 64, 3), ("f32", 64, 1), ("f32", 256, 5), ("bf16", 96, 40)])
def test_prompt_queries_that_weigh_nothing(gpu_lib, dtype, D, G, bad):
    """Queries of lse -infinity or +infinity weigh nothing whatever they hold, also
    where a tile's further rows are copies of the last one."""
    import torch
    rng = np.random.default_rng(G)
    n, H = 300, 2
    (q, k, v), host = ph.inputs(rng, n, H * G, H, D, dtype)
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32([0, n]), return_lse=True)
    for rows, value in ((n - 1, -np.inf), (slice(20, 23), np.inf), (slice(130, 150), -np.inf), ((200, H * G - 1), -np.inf)):
        lse[rows], q[rows] = value, bad
    want = ob.prompt_weights(*host[:2], lse.double().cpu().numpy(), [0, n], D ** -0.5, n)
    got = gpu_lib.prompt_weights(q, k, lse, _i32([0, n]), n)
    _weights_close(got, want, D)
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("dtype,D,H,G,n", [("bf16", 128, 1, 4, 2500), ("bf16", 256, 1, 2, 1111), ("f32", 64, 2, 1, 901)])
def test_long_prompt_weights(gpu_lib, dtype, D, H, G, n):
    """Against 64 bits on the device: the weights of long prompts, to 1e-6 of
    each (their sums have many terms, which the kernel adds in parts)."""
    import torch
    rng = np.random.default_rng(n)
    (q, k, v), _ = ph.inputs(rng, n, H * G, H, D, dtype)
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32([0, n]), return_lse=True)
    got = gpu_lib.prompt_weights(q, k, lse, _i32([0, n]), n).double()
    want, slack = torch.zeros_like(got), torch.zeros_like(got)
    seen = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
    for hq in range(H * G):
        qq, kk = q[:, hq].double().contiguous(), k[:, hq // G].double().t().contiguous()
        s, l = D ** -0.5 * (qq @ kk), lse[:, hq].double()[:, None]
        e = torch.exp(s - l).masked_fill(~seen, 0.0)
        big = D ** -0.5 * (qq.abs() @ kk.abs())
        want[0, hq // G] += e.sum(0)
        slack[0, hq // G] += (e * (ph.score_error(big, D) + 4 * U * (l.abs() + s.abs()))).sum(0)
    # a lane adds 32 terms, then the tiles' sums with their rounding kept
    assert ((got - want).abs() <= 1.01 * slack + 48 * U * want).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_weights_of_many_blocks_in_order(gpu_lib, dtype):
    """64 ragged sequences, some empty, of more blocks than the card takes at
    once: each block's weights once, the same bits as found the other way."""
    import torch
    rng = np.random.default_rng(17)
    lens = rng.integers(0, 400, 64)
    lens[[0, 20, 21, 63]] = 0
    starts = 1 + np.concatenate([[0], np.cumsum(lens)])
    T, H, cap = int(starts[-1]) + 2, 32, 300
    assert (-(-T // 128) + 64) * H >= 4096
    (q, k, v), host = ph.inputs(rng, T, H, H, 64, dtype)
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    got = gpu_lib.prompt_weights(q, k, lse, _i32(starts), cap)
    more = gpu_lib.prompt_weights(q, k, lse, _i32(np.concatenate([starts, [starts[-1]] * 9])), cap)
    assert torch.equal(got, more[:64]) and not more[64:].any()
    for b in (1, 40, 62):
        rows = slice(starts[b], starts[b + 1])
        want = ob.prompt_weights(host[0][rows, :2], host[1][rows, :2], lse[rows, :2].double().cpu().numpy(), [0, lens[b]], 0.125, cap)
        _weights_close(got[b:b + 1, :2], want, 64)
    fit = lens <= cap  # every query gives a weight of 1
    np.testing.assert_allclose(got.sum(2).cpu().numpy()[fit], np.outer(lens[fit], np.ones(H)), rtol=2e-3)


def test_prompt_weights_of_many_sequences(gpu_lib):
    """700 sequences, most of them empty or short: the same bits as in groups of 50."""
    import torch
    rng = np.random.default_rng(18)
    lens = rng.integers(0, 4, 700) * rng.integers(0, 2, 700)
    lens[[3, 300, 699]] = 200, 140, 33
    starts = np.concatenate([[0], np.cumsum(lens)])
    (q, k, v), host = ph.inputs(rng, int(starts[-1]), 4, 2, 64, "bf16")
    _, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    got = gpu_lib.prompt_weights(q, k, lse, _i32(starts), 180)
    for b in range(0, 700, 50):
        rows = slice(starts[b], starts[b + 50])
        part = gpu_lib.prompt_weights(q[rows], k[rows], lse[rows], _i32(starts[b:b + 51] - starts[b]), 180)
        assert torch.equal(got[b:b + 50], part)
    assert not got[torch.from_numpy(lens == 0)].any()
    _weights_close(got, ob.prompt_weights(*host[:2], lse.double().cpu().numpy(), starts, 0.125, 180), 64)


# --------------------------------------------------------------- nodes --
NODES = [  # fmt, dtype, P, H, G, D, N, lens, path
    ("e4m3", "bf16", 16, 2, 4, 128, 1, [0, 1, 15, 16, 17, 200], False),
    ("int8", "bf16", 32, 1, 1, 64, 5, [0, 63, 64, 65], True),
    ("e4m3", "bf16", 64, 2, 2, 96, 33, [0, 300, 64], True),
    ("int8", "f32", 128, 1, 8, 128, 9, [1, 127, 129, 700], True),
    ("e4m3", "f32", 16, 3, 3, 64, 17, [40, 5], False),
    ("int8", "bf16", 64, 1, 7, 256, 12, [0, 100, 65], True),
    ("e4m3", "f32", 128, 1, 2, 256, 64, [130], False),
    ("int8", "f32", 32, 2, 1, 96, 3, [31, 33], True),
    ("e4m3", "bf16", 64, 1, 40, 128, 64, [70], False),
]


def _nodes(gpu_lib, rng, fmt, dtype, P, H, G, D, N, lens, path):
    import torch
    B = len(lens)
    c, table = kh.make_cache(rng, fmt, lens, P, H, D, extra=N)
    x = torch.from_numpy(rng.normal(size=(B, N, H * G + H, D)).astype(np.float32)).to(_dt(dtype))
    q, k = x.cuda().split((H * G, H), 2)
    host = x.double().numpy()
    index = None
    if path:
        index = np.stack([np.concatenate([np.sort(rng.permutation(N)[:rng.integers(0, N + 1)]), np.full(N, -1)])[:N]
                          for _ in lens])
        index[0, :] = np.arange(N)
    weights = rng.random((B, H, table.shape[1] * P + 3)).astype(np.float32)
    # statistics as an attention gives them: some weights near 1, most small
    lse = np.abs(rng.normal(size=(B, N, H * G)) * 3 + 4).astype(np.float32)
    return c, table, q, k, (host[:, :, :H * G], host[:, :, H * G:]), index, weights, lse


@pytest.mark.parametrize("fmt,dtype,P,H,G,D,N,lens,path", NODES)
def test_node_weights(gpu_lib, fmt, dtype, P, H, G, D, N, lens, path):
    import torch
    rng = np.random.default_rng(P + D + N)
    c, table, q, k, host, index, weights, lse = _nodes(gpu_lib, rng, fmt, dtype, P, H, G, D, N, lens, path)
    lse[0, N // 2, 0] = -np.inf
    dev = kh.to_device(gpu_lib, c)
    counts = rng.integers(-1, N + 2, len(lens))
    for cnt, new in ((None, k), (counts, k), (None, None)):
        args = (dev, _i32(table), q, _f32(lse), _i32(lens))
        kw = dict(counts=None if cnt is None else _i32(cnt), index=None if index is None else _i32(index))
        w, out = _f32(weights), torch.full(weights.shape, 7.0, device="cuda")
        assert gpu_lib.kv_weights(*args, w, new, out=out, **kw) is out
        assert torch.equal(w, _f32(weights))
        want, written = ob.kv_weights(c, table, host[0], lse.astype(np.float64), lens, weights, D ** -0.5,
                                      None if new is None else host[1], cnt, index)
        rows = np.broadcast_to(written[:, None], weights.shape)
        _weights_close(out, want, D, rows)
        assert (out.cpu().numpy()[~rows] == 7.0).all()
        assert gpu_lib.kv_weights(*args, w, new, **kw) is w   # in place
        assert torch.equal(w[torch.from_numpy(rows.copy())], out[torch.from_numpy(rows.copy())])
        np.testing.assert_array_equal(w.cpu().numpy()[~rows], weights[~rows])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("fmt,dtype,G,D,N", [("e4m3", "bf16", 3, 128, 7), ("int8", "f32", 1, 64, 33), ("e4m3", "bf16", 2, 256, 2)])
def test_node_queries_that_weigh_nothing(gpu_lib, fmt, dtype, G, D, N, bad):
    """Nodes that no one looked at (lse -infinity, as an attention gives those past
    num_nodes) and whose queries are anything weigh nothing, the last ones too,
    whose rows fill up the block."""
    import torch
    rng = np.random.default_rng(N)
    c, table, q, k, host, _, weights, lse = _nodes(gpu_lib, rng, fmt, dtype, 32, 2, G, D, N, [70, 0, 33], False)
    lse[0, N - 1], lse[1, N // 2, G], lse[2] = -np.inf, np.inf, -np.inf
    want, written = ob.kv_weights(c, table, host[0], lse.astype(np.float64), [70, 0, 33], weights, D ** -0.5, host[1])
    q[0, N - 1] = q[1, N // 2, G] = q[2] = bad
    got = gpu_lib.kv_weights(kh.to_device(gpu_lib, c), _i32(table), q, _f32(lse), _i32([70, 0, 33]), _f32(weights), k)
    _weights_close(got, want, D, np.broadcast_to(written[:, None], weights.shape))
    assert torch.isfinite(got).all()


def test_node_weights_read_no_free_memory(gpu_lib):
    """Free slots, pages and table entries hold NaN (make_cache's poison), as
    do the nodes that are not kept; positions without a page gather nothing."""
    import torch
    rng = np.random.default_rng(4)
    c, table, q, k, host, _, weights, lse = _nodes(gpu_lib, rng, "e4m3", "bf16", 16, 2, 2, 128, 6, [100, 33], False)
    table[0, 2] = -1
    table[1, 0] = c["k_pages"].shape[0] + 3
    index = np.array([[0, 3, 6, 1, 2, 0], [5, 0, -1, 0, 0, 0]])
    q[0, [1, 2, 4, 5]] = q[1, 1:5] = k[0, [1, 2, 4, 5]] = k[1, 1:5] = float("nan")
    lse[0, [1, 2, 4, 5]] = lse[1, 1:5] = np.nan
    got = gpu_lib.kv_weights(kh.to_device(gpu_lib, c), _i32(table), q, _f32(lse), _i32([100, 33]), _f32(weights), k,
                             index=_i32(index), scale=-0.2)
    want, written = ob.kv_weights(c, table, host[0], lse.astype(np.float64), [100, 33], weights, -0.2, host[1], None, index)
    _weights_close(got, want, 128, np.broadcast_to(written[:, None], weights.shape))
    assert torch.isfinite(got).all()


# ------------------------------------------------------------- evict --
EVICT = [  # fmt, P, H, D, lens, budget, recent, limit
    ("e4m3", 16, 2, 64, [0, 20, 21, 40, 100], 20, 4, 20),
    ("int8", 32, 1, 96, [64, 65, 200, 33], 33, 33, 64),
    ("e4m3", 64, 3, 128, [300, 64, 129], 65, 0, 65),
    ("int8", 128, 2, 256, [700, 260], 131, 1, 200),
    ("e4m3", 128, 1, 256, [257, 300], 256, 100, 256),
    ("int8", 16, 1, 64, [2000, 1023, 1025], 1, 0, 1),
    ("e4m3", 32, 1, 64, [1500, 5000], 1024, 1000, 1024),
    ("int8", 64, 2, 96, [1100], 1000, 0, 1000),
    ("e4m3", 64, 2, 128, [1000, 4000], 100, 7, 100),
    ("int8", 32, 2, 256, [900, 400], 70, 3, 70),
    ("e4m3", 128, 1, 128, [3000, 513], 140, 0, 140),
]


def _evict_state(rng, fmt, P, H, D, lens, budget):
    c, table = kh.make_cache(rng, fmt, lens, P, H, D, spare=len(lens) * -(-budget // P))
    used = {int(x) for b, n in enumerate(lens) for x in table[b, :-(-n // P)]}
    free = [p for p in range(c["k_pages"].shape[0]) if p not in used]
    new = rng.permutation(free)[:len(lens) * -(-budget // P)].reshape(len(lens), -1).astype(np.int32)
    weights = np.exp(3 * rng.normal(size=(len(lens), H, table.shape[1] * P + 5))).astype(np.float32)
    weights *= rng.random(weights.shape) > 0.1
    return c, table, new, weights


def _evict_check(gpu_lib, c, table, lens, weights, new, budget, recent, limit):
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_evict(dev, _i32(table), _i32(lens), _f32(weights), _i32(new), budget, recent, limit=limit,
                           return_kept=True)
    want = ob.evict(c, table, lens, weights, new, budget, recent, limit)
    for name, g, w in zip(("table", "lengths", "weights", "kept"), got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w, name)
    host = kh.to_host(dev, c["fmt"])
    for n in ("k_pages", "v_pages"):
        np.testing.assert_array_equal(kh.canonical(host[n], c["fmt"]), kh.canonical(c[n], c["fmt"]), n)
    for n in ("k_scales", "v_scales"):
        np.testing.assert_array_equal(host[n], c[n], n)
    return got


@pytest.mark.parametrize("fmt,P,H,D,lens,budget,recent,limit", EVICT)
def test_evict(gpu_lib, fmt, P, H, D, lens, budget, recent, limit):
    rng = np.random.default_rng(P + D + budget)
    c, table, new, weights = _evict_state(rng, fmt, P, H, D, lens, budget)
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, recent, limit)


@pytest.mark.parametrize("kind", ["equal", "zeros", "two", "nan", "negative", "subnormal", "infinite"])
def test_evict_ties_and_special_weights(gpu_lib, kind):
    """Of equal weights the lowest positions stay; 0 has one sign; NaN is below
    all, infinities are at the ends."""
    rng = np.random.default_rng(6)
    lens, budget, recent = [500, 90, 1300], 77, 10
    c, table, new, weights = _evict_state(rng, "e4m3", 16, 2, 64, lens, budget)
    pick = rng.random(weights.shape)
    if kind == "equal":
        weights[:] = 0.3
    elif kind == "zeros":
        weights = np.where(pick < 0.5, 0.0, -0.0).astype(np.float32)
    elif kind == "two":
        weights = np.where(pick < 0.1, 2.0, 1.0).astype(np.float32)
    elif kind == "nan":
        weights[pick < 0.97] = np.nan
    elif kind == "negative":
        weights = -weights
    elif kind == "subnormal":
        weights = (rng.integers(0, 50, weights.shape) * 1e-45).astype(np.float32)
    else:
        weights[pick < 0.02], weights[pick > 0.5] = np.inf, -np.inf
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, recent, budget)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_evict_scales_far_apart(gpu_lib, fmt):
    """Blocks of very different magnitude, of zeros, of any scale (not only
    powers of two), at both ends of the range, NaN codes, missing pages, and
    new pages that do not exist."""
    rng = np.random.default_rng(7)
    P, H, D, lens, budget = 16, 2, 64, [400, 300, 64], 70
    c, table, new, weights = _evict_state(rng, fmt, P, H, D, lens, budget)
    s = np.exp2(rng.integers(-130, 119, c["k_scales"].shape).astype(np.float64)).astype(np.float32)
    c["k_scales"], c["v_scales"] = s.copy(), s[::-1].copy()
    ids = table[0, :25]
    c["k_scales"][ids[::3]] = 0.0
    c["v_scales"][ids[1::4]] = np.float32(0.3)  # one factor for all of them, so that the values' maximum is exact
    c["k_pages"][ids[3]] = 0
    c["v_pages"][ids[4:6]] = 0
    if fmt == "e4m3":
        c["k_pages"][ids[7], :, 3, 5] = 0x7f
        c["v_pages"][ids[8], :, 5, 3] = 0xff
    table[0, 9] = -1
    table[1, 2] = c["k_pages"].shape[0]
    new[1, 2], new[0, 4] = -1, c["k_pages"].shape[0] + 1
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, 6, 65536)   # nothing is cut
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, 6, 200)


def test_evict_long_and_shared_pages(gpu_lib):
    """Long sequences whose first pages are shared: the shared pages stay."""
    rng = np.random.default_rng(8)
    lens, P, budget = [9000, 8000, 16], 64, 2100
    c, table, new, weights = _evict_state(rng, "int8", P, 1, 64, lens, budget)
    table[1, :50] = table[0, :50]
    before = c["k_pages"][table[0, :50]].copy()
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, 300, budget)
    np.testing.assert_array_equal(c["k_pages"][table[0, :50]], before)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_evict_a_page_that_a_table_holds_twice(gpu_lib, P):
    """Positions of the same page one after the other, in and out of order."""
    rng = np.random.default_rng(P)
    lens, budget = [12 * P, 7 * P - 3], 2 * P + 5
    c, table, new, weights = _evict_state(rng, "e4m3", P, 2, 96, lens, budget)
    table[0, 1:6] = table[0, 0]
    table[1, 3], table[0, 9] = table[1, 5], -1
    weights[:, :, ::3] = 0
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, 2, budget)
    weights[0, :, :4 * P:P // 2] = 1e9  # two a page, far apart
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, 2, budget)


@pytest.mark.parametrize("kind", ["any", "equal", "mostly zero", "two", "nan"])
@pytest.mark.parametrize("budget,recent", [(1500, 100), (33, 33), (16400, 0)])
def test_evict_rows_of_several_workgroups(gpu_lib, kind, budget, recent):
    """Rows of more than 16384 positions, which several workgroups share, and
    short ones beside them; with more equal leading digits than are listed."""
    rng = np.random.default_rng(len(kind) + budget)
    lens = [40001, 16384, 16385, 100, 32768]
    c, table, new, weights = _evict_state(rng, "e4m3", 128, 1, 64, lens, budget)
    pick = rng.random(weights.shape)
    if kind == "equal":
        weights[:] = 0.3
    elif kind == "mostly zero":
        weights = np.where(pick < 0.01, weights, 0.0).astype(np.float32)
    elif kind == "two":
        weights = np.where(pick < 0.7, 1.0, 1.0 + 2.0 ** -23).astype(np.float32)
    elif kind == "nan":
        weights[pick < 0.999] = np.nan
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, recent, budget)


@pytest.mark.parametrize("kind", ["any", "decaying", "equal", "ties behind", "two"])
def test_evict_rows_of_more_than_eight_workgroups(gpu_lib, kind):
    """Rows of 9 and 17 workgroups, more than keep each other's lists in registers:
    weights that fit the lists, that decay slowly (as flat attention's do) and do
    not, that are all the same, the same from the ninth workgroup on, and of two
    values."""
    rng = np.random.default_rng(len(kind))
    lens, budget, recent = [9 * 16384 - 77, 17 * 16384, 3000], 400, 33
    c, table, new, weights = _evict_state(rng, "int8", 128, 1, 64, lens, budget)
    n, at = weights.shape[2], np.arange(weights.shape[2])
    if kind == "decaying":
        weights[:] = np.log(n / (at + 1.0)) * (1 + 0.01 * rng.random(weights.shape))
    elif kind == "equal":
        weights[:] = 0.3
    elif kind == "ties behind":
        weights[:] = np.where(at < 8 * 16384 + 9000, 0.25 * (at % 500 == 3), 0.125)
    elif kind == "two":
        weights[:] = np.where(rng.random(weights.shape) < 0.002, 1.0 + 2.0 ** -23, 1.0)
    _evict_check(gpu_lib, c, table, lens, weights, new, budget, recent, budget)


def test_evict_workspace_is_taken(gpu_lib):
    """A given workspace of any contents serves as a new one does; one that is too small is replaced."""
    import torch
    rng = np.random.default_rng(11)
    lens, budget = [20000, 300], 100
    c, table, new, weights = _evict_state(rng, "int8", 64, 2, 64, lens, budget)
    args = (_i32(table), _i32(lens), _f32(weights), _i32(new), budget, 5)
    size = gpu_lib.kv_evict_workspace_size(kh.to_device(gpu_lib, c), 2, table.shape[1])
    assert size > 256
    first = gpu_lib.kv_evict(kh.to_device(gpu_lib, c), *args, return_kept=True)
    for ws in (torch.full((size,), 0xff, dtype=torch.uint8, device="cuda"), torch.zeros(16, dtype=torch.uint8, device="cuda")):
        again = gpu_lib.kv_evict(kh.to_device(gpu_lib, c), *args, return_kept=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ----------------------------------------------------------- together --
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "f32")])
def test_prompt_rounds_and_eviction_together(gpu_lib, fmt, dtype):
    """The calls as a server makes them: prompts packed, attended, their
    weights gathered and cached; rounds of draft nodes attended, verified,
    their weights added and the accepted paths cached; sequences past the limit
    cut, their old pages given to the next.  The attention over what stays is
    that of the oracle's cache, which goes through the same steps."""
    import torch
    rng = np.random.default_rng(9)
    B, H, G, D, P, N, budget, limit = 3, 2, 2, 64, 16, 6, 48, 60
    lens, pages, width = [70, 30, 59], 40, 6
    Hq, dt = H * G, _dt(dtype)
    cache = gpu_lib.KVCache.empty(pages, P, H, D, dtype=torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)
    for t in (cache.k_pages, cache.v_pages):
        t.view(torch.uint8).zero_()
    cache.k_scales.zero_(), cache.v_scales.zero_()
    host = kh.to_host(cache, fmt)
    host = {n: (x.copy() if isinstance(x, np.ndarray) else x) for n, x in host.items()}
    free = list(rng.permutation(pages))
    table = np.full((B, width), -1, np.int32)
    for b in range(B):
        for col in range(width):
            table[b, col] = free.pop()

    starts = np.concatenate([[0], np.cumsum(lens)])
    (q, k, v), _ = ph.inputs(rng, int(starts[-1]), Hq, H, D, dtype)
    out, lse = gpu_lib.prompt_attention(q, k, v, _i32(starts), return_lse=True)
    weights = gpu_lib.prompt_weights(q, k, lse, _i32(starts), width * P)
    pad = torch.zeros((2, B, max(lens), H, D), dtype=dt, device="cuda")
    for b in range(B):
        pad[0, b, :lens[b]], pad[1, b, :lens[b]] = k[starts[b]:starts[b + 1]], v[starts[b]:starts[b + 1]]
    length = gpu_lib.kv_append(cache, _i32(table), pad[0], pad[1], _i32([0] * B), counts=_i32(lens))
    okv.append(host, table, pad[0].double().cpu().numpy(), pad[1].double().cpu().numpy(), [0] * B, counts=lens)
    cuts = 0
    for step in range(4):
        x = torch.from_numpy(rng.normal(size=(B, N, Hq + 2 * H, D)).astype(np.float32)).to(dt)
        qn, kn, vn = x.cuda().split((Hq, H, H), 2)
        x64 = x.double().numpy()
        tab = _i32(table)
        out, lse = gpu_lib.kv_attention(cache, tab, qn, length, kn, vn, return_lse=True)
        want = okv.attention(host, table, x64[:, :, :Hq], length.cpu().numpy(), D ** -0.5, x64[:, :, Hq:Hq + H],
                             x64[:, :, Hq + H:])
        tol, _ = kh.attention_bounds(*want, D ** -0.5, D, dtype)
        assert (np.abs(out.double().cpu().numpy() - want[0]) <= tol).all()
        index = np.full((B, N), -1)
        for b in range(B):
            index[b, :rng.integers(1, N)] = 0
            n = int((index[b] == 0).sum())
            index[b, :n] = np.arange(n)
        old = weights.cpu().numpy()
        length_before = length.cpu().numpy()
        gpu_lib.kv_weights(cache, tab, qn, lse, length, weights, kn, index=_i32(index))
        want, written = ob.kv_weights(host, table, x64[:, :, :Hq], lse.double().cpu().numpy(), length_before, old,
                                      D ** -0.5, x64[:, :, Hq:Hq + H], None, index)
        _weights_close(weights, want, D, np.broadcast_to(written[:, None], old.shape))
        after = gpu_lib.kv_append(cache, tab, kn, vn, length, index=_i32(index))
        np.testing.assert_array_equal(after.cpu().numpy(), okv.append(host, table, x64[:, :, Hq:Hq + H],
                                                                       x64[:, :, Hq + H:], length_before, index=index))
        new = np.array([[free.pop() for _ in range(-(-budget // P))] for _ in range(B)], np.int32)
        w = weights.cpu().numpy()
        tab, length, weights = gpu_lib.kv_evict(cache, tab, after, weights, _i32(new), budget, 8, limit=limit)
        want = ob.evict(host, table, after.cpu().numpy(), w, new, budget, 8, limit)
        for g, x in zip((tab, length, weights), want):
            np.testing.assert_array_equal(g.cpu().numpy(), x)
        for b in range(B):  # pages that came free, and enough for the next round
            if length[b] == budget and after[b] > limit:
                cuts += 1
                free = [int(p) for p in table[b] if p >= 0] + free
                row = want[0][b]
            else:
                free = [int(p) for p in new[b]] + free
                row = table[b]
            for col in range(width):
                if row[col] < 0:
                    row[col] = free.pop()
            table[b] = row
    assert cuts >= 2
