"""The 8-bit paged cache on the GPU against the fp64 oracle: append (bit for
bit), read back (exact), attention (within derived bounds)."""
import numpy as np
import pytest

import kv_helpers as kh
from oracle import kv as okv
from oracle.tree import verify_tree_greedy

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rand(rng, shape, dtype, device="cuda"):
    """Device tensor and its exact fp64 values."""
    import torch
    t = torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(_dt(dtype))
    return t.to(device), t.double().numpy()


def _i32(a, device="cuda"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)


def _same_cache(got, want):
    for n in ("k_pages", "v_pages"):
        np.testing.assert_array_equal(kh.canonical(got[n], want["fmt"]), kh.canonical(want[n], want["fmt"]), n)
    for n in ("k_scales", "v_scales"):
        np.testing.assert_array_equal(got[n], want[n], n)


# ---------------------------------------------------------------- append --
APPEND = [  # fmt, dtype, P, H, D, N, lens
    ("e4m3", "bf16", 16, 2, 64, 1, [0, 1, 15, 16, 17]),
    ("int8", "f32", 16, 1, 96, 5, [0, 13, 14, 15, 16]),
    ("e4m3", "f32", 32, 3, 128, 33, [0, 31, 40]),
    ("int8", "bf16", 64, 2, 128, 200, [0, 1, 63, 64, 100]),
    ("e4m3", "bf16", 128, 1, 256, 300, [5, 127, 128]),
    ("int8", "f32", 128, 2, 256, 129, [0, 100]),
    ("e4m3", "f32", 64, 1, 256, 64, [0, 32]),
    ("int8", "bf16", 32, 4, 96, 64, [0, 7, 500]),
]


@pytest.mark.parametrize("fmt,dtype,P,H,D,N,lens", APPEND)
def test_append_is_exact(gpu_lib, fmt, dtype, P, H, D, N, lens):
    rng = np.random.default_rng(P * D + N)
    c, table = kh.make_cache(rng, fmt, lens, P, H, D, extra=N)
    (k, k64), (v, v64) = _rand(rng, (len(lens), N, H, D), dtype), _rand(rng, (len(lens), N, H, D), dtype)
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_append(dev, _i32(table), k, v, _i32(lens))
    want = okv.append(c, table, k64, v64, lens)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    _same_cache(kh.to_host(dev, fmt), c)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_counts_index_and_growth(gpu_lib, fmt):
    """Ragged counts, paths ended by -1 and by N, values that grow a begun
    block's scale by far (old codes become subnormal or 0) and values too
    small to move it."""
    rng = np.random.default_rng(3)
    lens, P, H, D, N = [3, 10, 30, 0, 31, 5, 17], 32, 2, 64, 9
    c, table = kh.make_cache(rng, fmt, lens, P, H, D, extra=N)
    k, v = rng.normal(size=(2, len(lens), N, H, D))
    k[0] *= 1e4
    k[1] *= 1e-6
    v[2] *= 2.0 ** 40
    v[4] = 0.0
    k[5] *= 2.0 ** -140          # subnormal inputs
    k, v = k.astype(np.float32), v.astype(np.float32)
    index = np.array([[0, 2, 5, -1, 7, 0, 0, 0, 0], [8, 7, 6, 5, 4, 3, 2, 1, 0], [1, 1, 1, 9, 0, 0, 0, 0, 0],
                      [-1] * 9, [0, 1, 2, 3, 4, 5, 6, 7, 8], [2, 2 ** 31 - 1, 0, 0, 0, 0, 0, 0, 0],
                      [4, 5, 6, -2 ** 31, 0, 0, 0, 0, 0]])
    counts = np.array([9, 4, 100, 9, 7, 9, -3])
    import torch
    for cnt, idx in ((counts, index), (None, index), (counts, None)):
        dev = kh.to_device(gpu_lib, c)
        host = {n: (x.copy() if isinstance(x, np.ndarray) else x) for n, x in c.items()}
        got = gpu_lib.kv_append(dev, _i32(table), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                                _i32(lens), counts=None if cnt is None else _i32(cnt),
                                index=None if idx is None else _i32(idx))
        want = okv.append(host, table, k.astype(np.float64), v.astype(np.float64), lens, cnt, idx)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        _same_cache(kh.to_host(dev, fmt), host)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_special_values(gpu_lib, fmt):
    """Infinite values saturate and do not count for the scale, NaN does
    neither, a block of zeros gets the smallest scale; ties round to even."""
    import torch
    P, H, D, N = 16, 1, 64, 20
    c, table = kh.make_cache(np.random.default_rng(0), fmt, [7], P, H, D, extra=N)
    k = np.zeros((1, N, H, D), np.float32)
    v = np.random.default_rng(1).normal(size=k.shape).astype(np.float32)
    v[0, 2, 0, 5], v[0, 3, 0, 6], v[0, 4, 0, 7], v[0, 12, 0, 0] = np.inf, -np.inf, np.nan, 3.4e38
    k[0, 10, 0, :] = np.arange(64) + 0.5
    k[0, 11, 0, 0] = okv.QMAX[fmt]
    dev = kh.to_device(gpu_lib, c)
    gpu_lib.kv_append(dev, _i32(table), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), _i32([7]))
    okv.append(c, table, k.astype(np.float64), v.astype(np.float64), [7])
    _same_cache(kh.to_host(dev, fmt), c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,N,D", [("e4m3", 3, 64), ("int8", 3, 96), ("e4m3", 40, 256)])
def test_append_keeps_nan_and_reads_no_padding(gpu_lib, fmt, N, D, dtype):
    """NaN codes of a begun block stay NaN when its scale grows, by a little
    and from 0 or next to nothing; tokens behind counts hold anything."""
    import torch
    rng = np.random.default_rng(33)
    lens, P, H = [7, 9, 31, 5], 32, 2
    c, table = kh.make_cache(rng, fmt, lens, P, H, D, extra=N)
    if fmt == "e4m3":
        for b, n in enumerate(lens):
            c["k_pages"][table[b, 0], :, n // 2], c["v_pages"][table[b, 0], :, 3, :n] = 127, 255
    for b, s in ((1, 0.0), (3, 2.0 ** -126)):
        c["k_scales"][table[b, 0]] = c["v_scales"][table[b, 0]] = s
    x = (rng.normal(size=(2, 4, N, H, D)) * 1e3).astype(np.float32)
    counts = np.array([N, 1, N - 1, 2])
    k, v = (torch.from_numpy(t).to(_dt(dtype)) for t in x)
    k64, v64 = k.double().numpy(), v.double().numpy()
    for t in (k, v):
        t[torch.arange(N) >= torch.from_numpy(counts)[:, None]] = float("nan")
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_append(dev, _i32(table), k.cuda(), v.cuda(), _i32(lens), counts=_i32(counts))
    want = okv.append(c, table, k64, v64, lens, counts)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    _same_cache(kh.to_host(dev, fmt), c)


@pytest.mark.parametrize("fmt,dtype,P,D", [("e4m3", "bf16", 128, 128), ("int8", "f32", 128, 128), ("e4m3", "f32", 64, 256),
                                           ("int8", "bf16", 32, 96), ("e4m3", "bf16", 64, 256)])
@pytest.mark.parametrize("N", [1, 2, 4, 5, 9, 13, 14, 22])
def test_append_few_tokens(gpu_lib, fmt, dtype, P, D, N):
    """Calls around the size up to which one wave does a block, at every
    offset in a group of four, across a page's end, with and without growth
    of a block that is all but full."""
    rng = np.random.default_rng(P + D + N)
    lens, H = [0, 1, 2, 3, P - 1, P - 2, P - 3, P, P - N // 2 - 1, P - 1, 2 * P - 2], 2
    c, table = kh.make_cache(rng, fmt, lens, P, H, D, extra=N)
    x = rng.normal(size=(2, len(lens), N, H, D)).astype(np.float32)
    x[:, 4:7] *= 300.0  # these blocks' scales grow
    x[:, 9] *= 2.0 ** 60
    import torch
    k, v = (torch.from_numpy(t).to(_dt(dtype)) for t in x)
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_append(dev, _i32(table), k.cuda(), v.cuda(), _i32(lens))
    want = okv.append(c, table, k.double().numpy(), v.double().numpy(), lens)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    _same_cache(kh.to_host(dev, fmt), c)


def test_append_long_index(gpu_lib):
    """An index of hundreds of tokens over many pages: any order, repeats, an
    end past the first 256, a missing page in the middle."""
    rng = np.random.default_rng(6)
    B, N, P, H, D = 4, 600, 16, 1, 64
    lens = [0, 7, 100, 31]
    c, table = kh.make_cache(rng, "int8", lens, P, H, D, extra=N)
    table[2, 30] = -1
    index = rng.integers(0, N, (B, N))
    index[0, 431], index[1, 599], index[3, 0] = -1, N, -5
    (k, k64), (v, v64) = _rand(rng, (B, N, H, D), "bf16"), _rand(rng, (B, N, H, D), "bf16")
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_append(dev, _i32(table), k, v, _i32(lens), index=_i32(index))
    want = okv.append(c, table, k64, v64, lens, index=index)
    assert got.cpu().numpy().tolist() == want.tolist() == [431, 606, 480, 31]
    _same_cache(kh.to_host(dev, "int8"), c)


@pytest.mark.parametrize("indexed", [False, True])
def test_append_several_pages_a_workgroup(gpu_lib, indexed):
    """More pages than a head has workgroups (1024): ends and missing pages
    before, in and behind a workgroup's three pages, and a short sequence."""
    rng = np.random.default_rng(26)
    B, N, P, H, D = 7, 40000, 16, 1, 64
    lens = [0, 7, 0, 33, 5, 0, 16]
    counts = np.array([N, N, 17001, N, N, 20, 0])
    c, table = kh.make_cache(rng, "int8", [n + k for n, k in zip(lens, counts)], P, H, D, poison=False)
    table[0, 1000], table[3, 48], table[4, 50] = -1, 10 ** 9, -7
    index = rng.integers(0, N, (B, N))
    index[1, 31000], index[2, 17000], index[3, 40], index[5, 3] = -1, N, -1, N
    (k, k64), (v, v64) = _rand(rng, (B, N, H, D), "bf16"), _rand(rng, (B, N, H, D), "bf16")
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_append(dev, _i32(table), k, v, _i32(lens), counts=_i32(counts),
                            index=_i32(index) if indexed else None)
    want = okv.append(c, table, k64, v64, lens, counts, index if indexed else None)
    ends = [16000, 31007, 17000, 73, 800, 3, 16] if indexed else [16000, 40007, 17001, 768, 800, 20, 16]
    assert got.cpu().numpy().tolist() == want.tolist() == ends
    _same_cache(kh.to_host(dev, "int8"), c)


def test_longest_append(gpu_lib):
    """2^24 tokens by index in the smallest pages, against the same tokens in
    order and in sixteen calls."""
    import torch
    N, P, D = 1 << 24, 16, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k = torch.randn((1, N, 1, D), generator=g, device="cuda", dtype=torch.bfloat16)
    v = k.roll(1, 3)
    table = torch.randperm(N // P, generator=g, device="cuda").int().view(1, -1)
    whole, pieces = (gpu_lib.KVCache.empty(N // P, P, 1, D, dtype=torch.int8) for _ in range(2))
    index = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda").view(1, N)
    after = gpu_lib.kv_append(whole, table, k, v, _i32([0]), index=index)
    assert int(after[0]) == N
    at = _i32([0])
    for i in range(0, N, N // 16):
        src = slice(N - i - N // 16, N - i)
        at = gpu_lib.kv_append(pieces, table, k[:, src].flip(1), v[:, src].flip(1), at)
    assert int(at[0]) == N
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        assert torch.equal(getattr(whole, name), getattr(pieces, name)), name


def test_append_without_pages(gpu_lib):
    """A missing or foreign page ends the tokens there; a full table, a
    negative and a too large length write nothing out of place."""
    rng = np.random.default_rng(4)
    P, H, D, N = 16, 2, 64, 40
    lens = [0, 0, 0, -5, 10 ** 6]
    c, _ = kh.make_cache(rng, "e4m3", [0] * 12, P, H, D, extra=P, poison=False)
    table = np.array([[0, 1, -1, 2], [3, 99, 4, 5], [-7, 6, 6, 6], [7, 8, 2 ** 31 - 1, 9], [10, 11, 10, 11]], np.int32)
    (k, k64), (v, v64) = _rand(rng, (5, N, H, D), "f32"), _rand(rng, (5, N, H, D), "f32")
    dev = kh.to_device(gpu_lib, c)
    got = gpu_lib.kv_append(dev, _i32(table), k, v, _i32(lens)).cpu().numpy()
    want = okv.append(c, table, k64, v64, lens)
    assert got.tolist() == want.tolist() == [32, 16, 0, 32, 64]
    _same_cache(kh.to_host(dev, "e4m3"), c)


def test_append_in_pieces_and_strided_rows(gpu_lib):
    """One token at a time and several, from the rows of a fused projection
    (K and V slices of wider rows), against the oracle's same calls."""
    rng = np.random.default_rng(5)
    B, P, H, D = 3, 16, 2, 128
    lens = np.array([0, 14, 31])
    c, table = kh.make_cache(rng, "int8", lens.tolist(), P, H, D, extra=40)
    dev, tab = kh.to_device(gpu_lib, c), _i32(table)
    cur = _i32(lens)
    for n in (1, 1, 5, 1, 17, 2):
        fused, f64 = _rand(rng, (B, n, 4 * H + 2 * H, D), "bf16")
        cur = gpu_lib.kv_append(dev, tab, fused[:, :, 4 * H:5 * H], fused[:, :, 5 * H:], cur)
        lens = okv.append(c, table, f64[:, :, 4 * H:5 * H], f64[:, :, 5 * H:], lens)
        np.testing.assert_array_equal(cur.cpu().numpy(), lens)
    _same_cache(kh.to_host(dev, "int8"), c)


# ------------------------------------------------------------------ read --
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,P,H,D", [("e4m3", 16, 3, 64), ("int8", 32, 1, 96), ("e4m3", 64, 2, 128),
                                       ("int8", 128, 2, 256)])
def test_read_is_exact(gpu_lib, fmt, P, H, D, dtype):
    rng = np.random.default_rng(P)
    lens = [0, 1, P - 1, P, P + 1, 3 * P + 5]
    c, table = kh.make_cache(rng, fmt, lens, P, H, D)
    dev = kh.to_device(gpu_lib, c)
    for T, starts in ((1, None), (2 * P + 3, None), (P, [0, 0, 5, 1, P, 2 * P + 7]),
                      (70, [-3, 1, 2 ** 31 - 1, P - 1, 10 * P, P + 1])):
        k, v = gpu_lib.kv_read(dev, _i32(table), _i32(lens), T, starts=None if starts is None else _i32(starts),
                               dtype=_dt(dtype))
        want = okv.read(c, table, lens, T, starts)
        np.testing.assert_array_equal(k.double().cpu().numpy(), want[0])
        np.testing.assert_array_equal(v.double().cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,P,D", [("e4m3", 128, 256), ("int8", 128, 96), ("e4m3", 64, 256), ("int8", 32, 128)])
def test_read_short_and_long(gpu_lib, fmt, P, D, dtype):
    """A few tokens, and ranges of whole pages on both sides of the length
    from which workgroups share a page, at every offset in a group of four."""
    rng = np.random.default_rng(P + D)
    lens = [0, 5 * P, 4 * P + 3, P + 1, 6 * P - 1]
    c, table = kh.make_cache(rng, fmt, lens, P, 2, D)
    dev = kh.to_device(gpu_lib, c)
    for T, starts in ((1, [0, 5, P - 1, P, 6 * P - 2]), (3, [0, P - 2, 2, 1, P - 1]), (10, [1, P - 5, 2, P - 9, 3]),
                      (4 * P - 1, [0, 1, 2, 3, P - 1]), (4 * P, [3, 0, 2, 1, 2 * P - 1]), (5 * P + 2, [0, 1, 2, 3, P + 2])):
        k, v = gpu_lib.kv_read(dev, _i32(table), _i32(lens), T, starts=_i32(starts), dtype=_dt(dtype))
        want = okv.read(c, table, lens, T, starts)
        np.testing.assert_array_equal(k.double().cpu().numpy(), want[0])
        np.testing.assert_array_equal(v.double().cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,D,N", [("e4m3", 64, 5), ("int8", 96, 5), ("e4m3", 256, 70), ("int8", 128, 70)])
def test_finite_values_read_back_finite(gpu_lib, fmt, D, N, dtype):
    """Values next to the type's largest, whose code times the scale is
    2^128, and next to its smallest: what was finite reads back finite and
    within half a step of the code, NaN (e4m3) stays NaN, and magnitudes past
    the range, under scales of the caller's own, are the largest value."""
    import torch
    rng = np.random.default_rng(27)
    P, H = 16, 1
    c, table = kh.make_cache(rng, fmt, [0, 0, 3], P, H, D, extra=N, poison=False)
    dt = _dt(dtype)
    big = float(torch.finfo(dt).max)
    x = rng.normal(size=(2, 3, N, H, D)).astype(np.float32)
    x[:, 0] *= 3e36
    x[:, 0, :, :, 0], x[:, 0, :, :, 1], x[:, 0, 1, 0, 2], x[:, 0, 3, 0, 5] = big, -big, 3.38e38, np.nan
    x[:, 1] *= 2.0 ** -130
    k, v = (torch.from_numpy(t).to(dt) for t in x)
    dev, tab = kh.to_device(gpu_lib, c), _i32(table)
    after = gpu_lib.kv_append(dev, tab, k.cuda(), v.cuda(), _i32([0, 0, 3]))
    want = okv.append(c, table, k.double().numpy(), v.double().numpy(), [0, 0, 3])
    _same_cache(kh.to_host(dev, fmt), c)

    def check(cache, c):
        got = gpu_lib.kv_read(cache, tab, after, 3 + N, dtype=dt)
        for g, w in zip(got, okv.read(c, table, want, 3 + N)):
            # fp64 holds code * scale; float has it exactly once it is in range
            w = torch.from_numpy(np.clip(w, -big, big)).float().to(dt)
            assert torch.equal(g.cpu().isnan(), w.isnan())
            assert torch.equal(g.cpu().nan_to_num(), w.nan_to_num())
        return got
    for g, w in zip(check(dev, c), (k, v)):
        fine = w[0].isfinite()
        assert g[0, :N].cpu()[fine].isfinite().all() and fine.sum() >= fine.numel() - 1
        assert (g[0, :N, :, 0] == big).all() and (g[0, :N, :, 1] == -big).all()
        if fmt == "e4m3":
            assert g[0, 3, 0, 5].isnan()
    for name in ("k_scales", "v_scales"):
        c[name][:] = np.float32(1.3 * 2.0 ** 121)
    if dtype == "f32":  # such products round once in float, and once more in bf16
        check(kh.to_device(gpu_lib, c), c)
    else:
        got = gpu_lib.kv_read(kh.to_device(gpu_lib, c), tab, after, 3 + N, dtype=dt)
        assert all(not g.isinf().any() for g in got)


def test_read_without_pages(gpu_lib):
    rng = np.random.default_rng(8)
    c, table = kh.make_cache(rng, "e4m3", [40, 40], 16, 2, 64)
    table[0, 1], table[1, 0] = -1, 10 ** 6
    k, v = gpu_lib.kv_read(kh.to_device(gpu_lib, c), _i32(table), _i32([10 ** 6, -2]), 50)
    want = okv.read(c, table, [table.shape[1] * 16, 0], 50)
    np.testing.assert_array_equal(k.double().cpu().numpy(), want[0])
    np.testing.assert_array_equal(v.double().cpu().numpy(), want[1])


# ------------------------------------------------------------- attention --
def _tree(rng, B, N, bad=False):
    par = np.array([[-1] + [int(rng.integers(0, n)) for n in range(1, N)] for _ in range(B)], np.int32)
    if bad and N > 3:
        par[0, 2], par[0, 3] = 7, -9
    return par


def _check_attention(sv, c, table, lens, q, k, v, scale, dtype, parents=None, nodes=None, lse=True, **kw):
    (qd, q64), (kd, k64), (vd, v64) = q, k, v
    dev = kw.pop("dev", None) or kh.to_device(sv, c)
    got, glse = sv.kv_attention(dev, _i32(table), qd, _i32(lens), kd, vd, scale=scale, return_lse=True,
                                parents=None if parents is None else _i32(parents),
                                num_nodes=None if nodes is None else _i32(nodes), **kw)
    out, wlse, mag, big, cnt = okv.attention(c, table, q64, lens, scale, k64, v64, parents, nodes)
    tol, tol_lse = kh.attention_bounds(out, wlse, mag, big, cnt, scale, q64.shape[-1], dtype)
    g, gl = got.double().cpu().numpy(), glse.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(g), np.isnan(out))
    np.testing.assert_array_equal(np.isfinite(gl), np.isfinite(wlse))
    err = np.where(np.isnan(out), 0.0, np.abs(g - out) - tol)
    assert (err <= 0).all(), (np.unravel_index(err.argmax(), err.shape), err.max())
    f = np.isfinite(wlse)
    assert (np.abs(gl[f] - wlse[f]) <= tol_lse[f]).all()
    return got, glse


ATTEND = [  # fmt, dtype, P, H, G, D, N, lens, tree
    ("e4m3", "bf16", 16, 2, 4, 128, 1, [0, 1, 63, 64, 65, 500], False),
    ("int8", "bf16", 32, 1, 8, 64, 5, [0, 31, 32, 33, 700], False),
    ("e4m3", "bf16", 64, 2, 4, 128, 9, [0, 5, 64, 300, 1030], False),
    ("int8", "bf16", 64, 2, 4, 128, 16, [0, 127, 129, 640], True),
    ("e4m3", "bf16", 128, 1, 7, 96, 13, [0, 100, 128, 400], True),
    ("int8", "bf16", 128, 1, 2, 256, 33, [0, 1, 255, 513], True),
    ("e4m3", "bf16", 64, 1, 3, 64, 64, [0, 70, 200], True),
    ("e4m3", "bf16", 32, 3, 1, 256, 7, [33, 64, 0], False),
    ("int8", "bf16", 16, 1, 16, 128, 64, [17, 90], True),
    ("e4m3", "f32", 16, 2, 4, 128, 3, [0, 1, 63, 64, 65, 500], False),
    ("int8", "f32", 64, 1, 8, 256, 9, [0, 31, 200], True),
    ("int8", "f32", 32, 4, 1, 64, 9, [0, 65, 300], False),
    ("e4m3", "f32", 128, 2, 3, 96, 40, [0, 129, 260], True),
]


@pytest.mark.parametrize("fmt,dtype,P,H,G,D,N,lens,tree", ATTEND)
def test_attention(gpu_lib, fmt, dtype, P, H, G, D, N, lens, tree):
    rng = np.random.default_rng(D + N + P)
    B = len(lens)
    c, table = kh.make_cache(rng, fmt, lens, P, H, D)
    q = _rand(rng, (B, N, H * G, D), dtype)
    k, v = _rand(rng, (B, N, H, D), dtype), _rand(rng, (B, N, H, D), dtype)
    par = _tree(rng, B, N, bad=True) if tree else None
    _check_attention(gpu_lib, c, table, lens, q, k, v, D ** -0.5, dtype, par)
    # the cached tokens alone: rows of empty sequences see nothing
    none = (None, None)
    got, lse = _check_attention(gpu_lib, c, table, lens, q, none, none, 0.3, dtype)
    for b, n in enumerate(lens):
        if n == 0:
            assert (got[b] == 0).all() and (lse[b] == -np.inf).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_attention_every_block_of_queries(gpu_lib, D, dtype, fmt):
    """1 to 64 queries of a cached head: each kernel variant, full and partly
    filled blocks of 16, and every block of 16 nodes."""
    rng = np.random.default_rng(D)
    P, lens = 32, [150, 0, 64]
    c, table = kh.make_cache(rng, fmt, lens, P, 1, D)
    for N in (2, 16, 17, 32, 41, 48, 64):
        q, k, v = (_rand(rng, (3, N, 1, D), dtype) for _ in range(3))
        _check_attention(gpu_lib, c, table, lens, q, k, v, D ** -0.5, dtype, _tree(rng, 3, N) if N % 2 else None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_long_and_split(gpu_lib, dtype):
    """Few sequences with long caches next to short and empty ones: the
    length is split over many workgroups."""
    rng = np.random.default_rng(11)
    lens, P, H, D, N = [9000, 0, 3, 4097], 64, 1, 64, 2
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D)
    q = _rand(rng, (4, N, 2, D), dtype)
    k, v = _rand(rng, (4, N, H, D), dtype), _rand(rng, (4, N, H, D), dtype)
    _check_attention(gpu_lib, c, table, lens, q, k, v, 0.125, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_sharp_scores(gpu_lib, dtype):
    """Scores of +-hundreds: one token carries almost all weight, and the
    maximum grows along the sequence."""
    rng = np.random.default_rng(12)
    lens, P, H, D, N = [300, 129], 32, 2, 128, 4
    c, table = kh.make_cache(rng, "int8", lens, P, H, D)
    q = _rand(rng, (2, N, 4, D), dtype)
    k, v = _rand(rng, (2, N, H, D), dtype), _rand(rng, (2, N, H, D), dtype)
    _check_attention(gpu_lib, c, table, lens, q, k, v, 20.0, dtype)
    _check_attention(gpu_lib, c, table, lens, q, k, v, -3.0, dtype)
    _check_attention(gpu_lib, c, table, lens, q, k, v, 0.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_ragged_nodes(gpu_lib, dtype):
    rng = np.random.default_rng(13)
    lens, P, H, D, N = [70, 0, 16, 33, 5], 16, 2, 64, 12
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D)
    q = _rand(rng, (5, N, 6, D), dtype)
    k, v = _rand(rng, (5, N, H, D), dtype), _rand(rng, (5, N, H, D), dtype)
    nodes = [12, 0, -4, 7, 99]
    for par in (None, _tree(rng, 5, N)):
        got, lse = _check_attention(gpu_lib, c, table, lens, q, k, v, 0.125, dtype, par, nodes)
        for b, n in enumerate([12, 0, 0, 7, 12]):
            assert (got[b, n:] == 0).all() and (lse[b, n:] == -np.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [6, 40])
def test_attention_nan_and_infinity_in_unseen_nodes(gpu_lib, dtype, N):
    """NaN, infinities and the type's largest values in nodes reach exactly
    the queries that see them."""
    import torch
    rng = np.random.default_rng(14)
    lens, P, H, D = [50, 0, 17], 16, 2, 64
    c, table = kh.make_cache(rng, "int8", lens, P, H, D)
    q, k, v = (_rand(rng, (3, N, h, D), dtype) for h in (4, H, H))
    par = _tree(rng, 3, N)
    par[:, 3], par[:, 4], par[:, 5] = 1, 0, 0
    see = np.stack([okv.node_sets(par[b], N) for b in range(3)])
    dev = kh.to_device(gpu_lib, c)
    args = (dev, _i32(table))
    clean = gpu_lib.kv_attention(*args, q[0], _i32(lens), k[0], v[0], parents=_i32(par))
    big = float(torch.finfo(_dt(dtype)).max)
    for val in (float("nan"), float("inf"), -float("inf"), big, -big):
        for where in ("k", "v"):
            kk, vv = k[0].clone(), v[0].clone()
            (kk if where == "k" else vv)[:, 3, :, 7] = val
            got = gpu_lib.kv_attention(*args, q[0], _i32(lens), kk, vv, parents=_i32(par))
            blind = torch.from_numpy(~see[:, :, 3]).cuda()
            assert torch.equal(got[blind], clean[blind]), (val, where)
            if val != val:
                seen = got[~blind]
                assert (seen.isnan().any(-1) if where == "v" else seen.isnan().all(-1)).all()
            elif where == "v" and abs(val) == float("inf"):
                assert (got[~blind][..., 7] == val).all() and got[~blind][..., :7].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N,lens", [(64, 1, [50, 7000, 16]), (128, 17, [0, 50, 5000]), (256, 40, [0, 70, 9])])
def test_attention_nodes_with_the_lowest_score(gpu_lib, D, N, lens, dtype):
    """A key at the type's lowest value, whose score passes 32 bits downwards,
    has a weight of 0 where it is seen, as a key far below the others has:
    alone in its wave's block of nodes, beside others, under a tree."""
    import torch
    rng = np.random.default_rng(28)
    P, H = 32, 2
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D)
    (q, _), (k, _), (v, v64) = (_rand(rng, (3, N, h, D), dtype) for h in (4, H, H))
    q[..., 7] = 8.0
    low = N - 1  # the only node of its block that the last queries see, for 17 nodes
    par = _tree(rng, 3, N) if N == 40 else None
    res = []
    for val in (-20000.0, float(torch.finfo(_dt(dtype)).min)):
        k[:, low, :, 7] = val
        if val == -20000.0:
            res.append(_check_attention(gpu_lib, c, table, lens, (q, q.double().cpu().numpy()),
                                        (k, k.double().cpu().numpy()), (v, v64), 1.0, dtype, par))
        else:
            res.append(gpu_lib.kv_attention(kh.to_device(gpu_lib, c), _i32(table), q, _i32(lens), k, v, scale=1.0,
                                            return_lse=True, parents=None if par is None else _i32(par)))
    for a, b in zip(*res):
        assert a.isfinite().all() and torch.equal(a, b)
    # alone, nothing weighs anything: as a query that sees nothing
    out, lse = gpu_lib.kv_attention(kh.to_device(gpu_lib, c), _i32(table), q[:, low:].contiguous(), _i32([0, 0, 0]),
                                    k[:, low:].contiguous(), v[:, low:].contiguous(), scale=1.0, return_lse=True)
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,D", [("e4m3", 64), ("int8", 256)])
def test_attention_smallest_key_scales(gpu_lib, fmt, D, dtype):
    """Queries next to 2^100 over blocks of the smallest K scales, and a scale
    of 0 or next to it: scores are what they are, however small their factor."""
    rng = np.random.default_rng(29)
    lens, P, H, N = [24, 9], 16, 1, 3
    c, table = kh.make_cache(rng, fmt, lens, P, H, D)
    q, q64 = _rand(rng, (2, N, 4, D), dtype)
    q, q64 = q * 2.0 ** 97, q64 * 2.0 ** 97
    none = (None, None)
    for k_scale in (2.0 ** -126, 2.0 ** -140, 0.0):
        c["k_scales"][table[0, :2]] = c["k_scales"][table[1, 0]] = k_scale
        for scale in (0.125, 2.0 ** -12, -(2.0 ** -14), 0.0):
            _check_attention(gpu_lib, c, table, lens, (q, q64), none, none, scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_attention_keeps_nan_of_tiny_blocks(gpu_lib, D, dtype):
    """NaN appended among zeros, among values next to nothing and as a whole
    block reaches every query, in its channels only; NaN in the slots behind
    the last token reaches none."""
    import torch
    rng = np.random.default_rng(30)
    P, H, N, T = 32, 2, 3, 120
    lens = [T, 70, 33, 1]
    c, table = kh.make_cache(rng, "e4m3", [0] * 4, P, H, D, extra=T)
    (k, k64), (v, _) = _rand(rng, (4, T, H, D), dtype), _rand(rng, (4, T, H, D), dtype)
    v[0, 32:64], v[0, 64:96] = 0.0, 2.0 ** -110
    v[0, 40, 0, 5], v[0, 47, 1, 6], v[0, 64, 1, D - 1] = np.nan, np.nan, np.nan
    v[1, 64:], v[2, 32:], v[3] = np.nan, 0.0, 0.0
    v[2, 32, 0, 17] = np.nan
    v64 = v.double().cpu().numpy()
    dev, tab = kh.to_device(gpu_lib, c), _i32(table)
    after = gpu_lib.kv_append(dev, tab, k, v, _i32([0] * 4), counts=_i32(lens))
    assert after.tolist() == okv.append(c, table, k64, v64, [0] * 4, lens).tolist() == lens
    q = _rand(rng, (4, N, 8, D), dtype)
    kn, vn = _rand(rng, (4, N, H, D), dtype), _rand(rng, (4, N, H, D), dtype)
    for new in ((kn, vn), ((None, None), (None, None))):
        out, _ = _check_attention(gpu_lib, c, table, lens, q, *new, D ** -0.5, dtype, dev=dev)
        nan = out.isnan().all(1)  # [sequence, head, channel]: every node
        assert torch.equal(nan, out.isnan().any(1))
        want = torch.zeros_like(nan)
        want[0, :4, 5], want[0, 4:, 6], want[0, 4:, D - 1], want[1], want[2, :4, 17] = True, True, True, True, True
        assert torch.equal(nan, want)


def test_attention_bad_pages_and_lengths(gpu_lib):
    """Positions without a page are not seen; lengths are clamped."""
    rng = np.random.default_rng(15)
    lens, P, H, D, N = [200, 200, 200, 200], 16, 2, 64, 3
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D)
    table[0, 2], table[1, 12], table[2, :] = -1, 2 ** 31 - 1, -1
    q, k, v = (_rand(rng, (4, N, h, D), "f32") for h in (4, H, H))
    # a length past the table is clamped to it: the free slots it then reaches hold NaN here
    _check_attention(gpu_lib, c, table, [10 ** 9, 200, 200, -1], q, k, v, 0.125, "f32")
    full, ftab = kh.make_cache(rng, "e4m3", [14 * P] * 4, P, H, D, poison=False)
    _check_attention(gpu_lib, full, ftab[:, :14], [10 ** 9, 14 * P, 0, -1], q, k, v, 0.125, "f32")
    _check_attention(gpu_lib, c, table, [200, 200, 200, 0], q, (None, None), (None, None), 0.125, "f32")


def test_attention_arbitrary_scales_and_shared_pages(gpu_lib):
    """Scales that are no powers of two, and a prefix that two sequences share."""
    rng = np.random.default_rng(16)
    lens, P, H, D, N = [100, 100], 32, 2, 128, 3
    c, table = kh.make_cache(rng, "int8", lens, P, H, D)
    c["k_scales"] = (c["k_scales"] * 1.37).astype(np.float32)
    c["v_scales"] = (c["v_scales"] * 0.71).astype(np.float32)
    table[1, :3] = table[0, :3]
    q, k, v = (_rand(rng, (2, N, h, D), "bf16") for h in (4, H, H))
    _check_attention(gpu_lib, c, table, lens, q, k, v, 0.1, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_blocks_of_zeros(gpu_lib, fmt, dtype):
    """Blocks of zeros, which have the smallest scale, keep their weight in
    the sums: next to other blocks, alone, as keys and as values; so do scales
    of 0 and tiny ones."""
    rng = np.random.default_rng(24)
    lens, P, H, D, N = [300, 200, 64, 130], 32, 2, 64, 3
    c, table = kh.make_cache(rng, fmt, lens, P, H, D)
    zero = [table[0, 1], table[0, 4], table[0, 9], *table[1, :7], table[2, 0]]
    for name in ("k", "v"):
        c[name + "_pages"][zero] = 0
        c[name + "_scales"][zero] = 2.0 ** -126
    c["v_scales"][table[2, 1]] = 0.0
    c["k_scales"][table[3, 0]] = 0.0
    c["v_scales"][table[3, 2]] = 2.0 ** -80
    q, k, v = (_rand(rng, (4, N, h, D), dtype) for h in (8, H, H))
    _check_attention(gpu_lib, c, table, lens, q, k, v, D ** -0.5, dtype)
    out, lse = _check_attention(gpu_lib, c, table, lens, q, (None, None), (None, None), D ** -0.5, dtype)
    assert (out[1] == 0).all()
    np.testing.assert_allclose(lse[1].cpu().numpy(), np.log(200.0), rtol=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_fused_rows_and_repeatability(gpu_lib, dtype):
    """q, k and v as slices of one projection's rows give the bits of
    contiguous copies, twice."""
    import torch
    rng = np.random.default_rng(17)
    lens, P, H, G, D, N = [1000, 0, 77], 64, 2, 4, 128, 5
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32(lens)
    fused, _ = _rand(rng, (3, N, H * G + 2 * H, D), dtype)
    q, k, v = fused[:, :, :H * G], fused[:, :, H * G:H * G + H], fused[:, :, H * G + H:]
    a = gpu_lib.kv_attention(dev, tab, q, ln, k, v, return_lse=True)
    for _ in range(3):
        b = gpu_lib.kv_attention(dev, tab, q.contiguous(), ln, k.contiguous(), v.contiguous(), return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = gpu_lib.kv_attention(dev, tab, q[:, :1], ln, k[:, :1], v[:, :1])  # N = 1: rows far apart
    assert torch.equal(one, gpu_lib.kv_attention(dev, tab, q[:, :1].contiguous(), ln, k[:, :1].contiguous(),
                                                 v[:, :1].contiguous()))


def test_other_stream_and_graph(gpu_lib):
    """Attention, append and read on a side stream, then captured into one
    graph and replayed between eager work; every replay gives the eager bits."""
    import torch
    rng = np.random.default_rng(18)
    lens, P, H, D, N = [130, 5], 16, 2, 64, 4
    c, table = kh.make_cache(rng, "int8", lens, P, H, D, extra=N)
    q, k, v = (_rand(rng, (2, N, h, D), "bf16")[0] for h in (4, H, H))
    tab, ln = _i32(table), _i32(lens)

    def step(dev, ws):
        out, lse = gpu_lib.kv_attention(dev, tab, q, ln, k, v, return_lse=True, workspace=ws)
        after = gpu_lib.kv_append(dev, tab, k, v, ln)
        return (out, lse, after) + gpu_lib.kv_read(dev, tab, after, 140)

    dev = kh.to_device(gpu_lib, c)
    ws = torch.empty(gpu_lib.kv_attention_workspace_size(dev, 2, N, 4, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    want = [t.clone() for t in step(kh.to_device(gpu_lib, c), ws)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(dev, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the append may have rounded the begun blocks again; from here on the same call changes nothing
    want = [t.clone() for t in step(dev, ws)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(dev, ws)
    for _ in range(4):
        for t in outs:
            t.fill_(1)
        ws.fill_(0xff)
        graph.replay()
        eager = step(dev, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, want))


def test_graph_owns_its_workspace(gpu_lib):
    """A captured call that allocates its own workspace, parts joined by a
    second launch, two graphs replayed in turn."""
    import torch
    rng = np.random.default_rng(20)
    lens, P, H, D, N = [5000, 3], 32, 1, 64, 2
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32(lens)
    qs = [_rand(rng, (2, N, 4, D), "f32")[0] for _ in range(2)]
    want = [gpu_lib.kv_attention(dev, tab, q, ln) for q in qs]
    assert gpu_lib.kv_attention_workspace_size(dev, 2, N, 4, table.shape[1]) > 256
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gpu_lib.kv_attention(dev, tab, q, ln))
        graphs.append(g)
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            assert torch.equal(gpu_lib.kv_attention(dev, tab, qs[0], ln), want[0])
            torch.cuda.synchronize()
            assert torch.equal(o, w)


def test_two_streams_at_once(gpu_lib):
    """Two calls in flight together on two streams, each with its own workspace."""
    import torch
    rng = np.random.default_rng(21)
    lens, P, H, D, N = [9000, 2000, 0], 64, 2, 128, 4
    c, table = kh.make_cache(rng, "int8", lens, P, H, D)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32(lens)
    qs = [_rand(rng, (3, N, 8, D), "bf16")[0] for _ in range(2)]
    want = [gpu_lib.kv_attention(dev, tab, q, ln) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(gpu_lib.kv_attention(dev, tab, qs[i], ln))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_largest_batch(gpu_lib):
    """65535 sequences: the first and the last give what small batches give."""
    import torch
    B, P, H, D = 65535, 16, 1, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cache = gpu_lib.KVCache.empty(B, P, H, D, dtype=torch.int8)
    for t in (cache.k_pages, cache.v_pages):
        t.zero_()
    cache.k_scales.fill_(1), cache.v_scales.fill_(1)
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    lens = (torch.arange(B, device="cuda") % 14).int()
    k, v, q = (torch.randn((B, 2, h, D), generator=g, device="cuda") for h in (H, H, 2))
    after = gpu_lib.kv_append(cache, table, k, v, lens)
    assert torch.equal(after, lens + 2)
    rk, rv = gpu_lib.kv_read(cache, table, after, P, dtype=torch.float32)
    out = gpu_lib.kv_attention(cache, table, q, after, k, v)
    for s in (slice(0, 50), slice(B - 50, B)):
        a, b = gpu_lib.kv_read(cache, table[s].contiguous(), after[s].contiguous(), P, dtype=torch.float32)
        assert torch.equal(a, rk[s]) and torch.equal(b, rv[s])
        o = gpu_lib.kv_attention(cache, table[s].contiguous(), q[s].contiguous(), after[s].contiguous(),
                                 k[s].contiguous(), v[s].contiguous())
        assert torch.equal(o, out[s])
        n = lens[s].long()[:, None] + torch.arange(2, device="cuda")
        got = rk[s].gather(1, n[:, :, None, None].expand(-1, -1, H, D))
        # an int8 code is off by half a step of its block's scale: a begun block keeps its scale of 1 here, since
        # 127 exceeds every value, and a fresh one has the smallest power of two from its largest value over 127 up
        step = cache.k_scales[s][:, None, :, None]
        assert ((got - k[s]).abs() <= step / 2).all()
        top = k[s].abs().amax((1, 2, 3))
        assert (torch.where(lens[s] > 0, cache.k_scales[s, 0] == 1,
                            (top <= 127 * cache.k_scales[s, 0]) & (top > 63.5 * cache.k_scales[s, 0]))).all()


def test_pool_past_32_bits(gpu_lib):
    """Pages more than 4 GiB into the pool hold and give what pages at its start do."""
    import torch
    rng = np.random.default_rng(22)
    P, H, D, N = 128, 8, 256, 300
    pages = (5 << 30) // (P * H * D)
    big = gpu_lib.KVCache.empty(pages, P, H, D)
    small = gpu_lib.KVCache.empty(3, P, H, D)
    (k, _), (v, _), (q, _) = (_rand(rng, (1, N, h, D), "bf16") for h in (H, H, 16))
    res = []
    for cache, table in ((big, [[pages - 1, pages - 3, pages - 2]]), (small, [[0, 2, 1]])):
        tab = _i32(table)
        n = gpu_lib.kv_append(cache, tab, k, v, _i32([0]))
        res.append((n,) + gpu_lib.kv_read(cache, tab, n, N) +
                   (gpu_lib.kv_attention(cache, tab, q[:, :4].contiguous(), n, k[:, :4].contiguous(),
                                         v[:, :4].contiguous()),))
    assert int(res[0][0]) == N and all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("G", [1000, 1024])
def test_largest_group_of_heads(gpu_lib, G):
    """Up to 65536 queries share a cached head: each gives what it gives alone."""
    import torch
    rng = np.random.default_rng(25)
    P, D, N = 32, 64, 64
    c, table = kh.make_cache(rng, "e4m3", [100], P, 1, D)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32([100])
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q = torch.randn((1, N, G, D), generator=g, device="cuda").bfloat16()
    (k, _), (v, _) = _rand(rng, (1, N, 1, D), "bf16"), _rand(rng, (1, N, 1, D), "bf16")
    out = gpu_lib.kv_attention(dev, tab, q, ln, k, v)
    for h in (0, G // 2, G - 8):
        assert torch.equal(gpu_lib.kv_attention(dev, tab, q[:, :, h:h + 8], ln, k, v), out[:, :, h:h + 8])


def test_misaligned_rows_are_refused(gpu_lib):
    import torch
    rng = np.random.default_rng(23)
    c, table = kh.make_cache(rng, "int8", [4], 16, 1, 64, extra=4)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32([4])
    flat = torch.zeros(2 * 64 + 4, device="cuda", dtype=torch.bfloat16)
    x = flat[4:].view(1, 2, 1, 64)
    for call in (lambda: gpu_lib.kv_append(dev, tab, x, x, ln), lambda: gpu_lib.kv_attention(dev, tab, x, ln, x, x)):
        with pytest.raises(gpu_lib.SpecVerifyError) as e:
            call()
        assert e.value.code == -6
    both = _i32([4, 0])
    with pytest.raises(ValueError):
        gpu_lib.kv_append(dev, tab, x.clone(), x.clone(), ln, out_lengths=ln)
    with pytest.raises(ValueError):
        gpu_lib.kv_append(dev, torch.cat((tab, tab)), torch.zeros(2, 1, 1, 64, device="cuda"),
                          torch.zeros(2, 1, 1, 64, device="cuda"), _i32([0, 0, 0])[:2], out_lengths=both.new_zeros(2)[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N,G", [(64, 5, 3), (128, 20, 4), (256, 33, 1)])
def test_padding_may_hold_anything(gpu_lib, D, N, G, dtype):
    """A padded batch: queries, keys and values of nodes that do not exist,
    and table columns behind a sequence's pages that name pages of NaN, reach
    no other query; a live query of NaN reaches itself only."""
    import torch
    rng = np.random.default_rng(32)
    P, H = 16, 2
    lens, nodes = [0, 33, 5000, 17, 100], [1, N, N - 2, 0, 3]
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D, spare=40)
    dev, ln, nn = kh.to_device(gpu_lib, c), _i32(lens), _i32(nodes)
    q, k, v = (_rand(rng, (5, N, h, D), dtype)[0] for h in (H * G, H, H))
    par = _i32(_tree(rng, 5, N))
    want = gpu_lib.kv_attention(dev, _i32(table), q, ln, k, v, parents=par, num_nodes=nn, return_lse=True)
    wild = table.copy()
    poisoned = np.setdiff1d(np.arange(c["k_pages"].shape[0]), table)
    for b, n in enumerate(lens):
        free = wild[b, (n + P - 1) // P:]
        free[:] = rng.choice(poisoned, free.shape)
    live = torch.arange(N, device="cuda") < nn[:, None]
    q2, k2, v2 = (torch.where(live[..., None, None], t, float("nan")) for t in (q, k, v))
    for val in (float("nan"), float("inf")):
        for t in (q2, k2, v2):
            t[~live] = val
        got = gpu_lib.kv_attention(dev, _i32(wild), q2, ln, k2, v2, parents=par, num_nodes=nn, return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (got[0][~live] == 0).all() and (got[1][~live] == -np.inf).all()
    q2 = q.clone()
    q2[1, N - 1, 1], q2[2, 0, 0] = float("nan"), float("inf")
    got = gpu_lib.kv_attention(dev, _i32(table), q2, ln, k, v, parents=par, num_nodes=nn, return_lse=True)
    hit = torch.zeros(got[1].shape, dtype=torch.bool, device="cuda")
    hit[1, N - 1, 1], hit[2, 0, 0] = True, True
    assert all(torch.equal(a[~hit], b[~hit]) for a, b in zip(got, want))
    assert got[0][hit].isnan().all()


def test_gradients_are_refused(gpu_lib):
    """Queries, keys or values that require gradients: the same values, and a
    backward pass through them raises."""
    import torch
    rng = np.random.default_rng(31)
    lens, P, H, D, N = [40, 5], 16, 2, 64, 3
    c, table = kh.make_cache(rng, "int8", lens, P, H, D)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32(lens)
    x = [_rand(rng, (2, N, h, D), "f32")[0] for h in (4, H, H)]
    want = gpu_lib.kv_attention(dev, tab, x[0], ln, *x[1:], return_lse=True)
    assert not any(t.requires_grad for t in want)
    for i in range(3):
        y = [t.clone().requires_grad_(j == i) for j, t in enumerate(x)]
        got = gpu_lib.kv_attention(dev, tab, y[0], ln, *y[1:], return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for t in (got[0], got[1], gpu_lib.kv_attention(dev, tab, y[0], ln, *y[1:])):
            with pytest.raises(NotImplementedError, match="forward only"):
                (t.sum() + y[i].sum()).backward()
        with torch.no_grad():
            assert not gpu_lib.kv_attention(dev, tab, y[0], ln, *y[1:]).requires_grad


def test_overlapping_lengths_are_refused(gpu_lib):
    """New lengths over a part of any array the call reads; beside it they are fine."""
    import torch
    B, N, P, D = 2, 3, 16, 64
    cache = gpu_lib.KVCache.empty(4, P, 1, D)
    x = torch.zeros(B, N, 1, D, device="cuda")
    buf = torch.zeros(64, dtype=torch.int32, device="cuda")
    table = buf[:8].view(B, 4)
    lengths, counts, index = buf[16:18], buf[24:26], buf[32:38].view(B, N)
    table.copy_(_i32([[0, 1, 9, 9], [2, 3, 9, 9]])), counts.fill_(2), index.copy_(_i32([[2, 1, 0]] * 2))
    for name, first, n in (("lengths", 16, 2), ("counts", 24, 2), ("index", 32, 6), ("page_table", 0, 8)):
        for at in {first, first + 1, first + n - 1, max(first - 1, 0)}:
            with pytest.raises(ValueError, match=f"overlap {name}"):
                gpu_lib.kv_append(cache, table, x, x, lengths, counts=counts, index=index, out_lengths=buf[at:at + 2])
        got = gpu_lib.kv_append(cache, table, x, x, lengths, counts=counts, index=index,
                                out_lengths=buf[first + n:first + n + 2])
        assert got.tolist() == [2, 2]


def test_verify_round_with_trees(gpu_lib):
    """A run of them together: prompts cached, then rounds of attention over
    a token tree, greedy verification of the logits its outputs give, and the
    accepted path appended straight from the verification's outputs."""
    import torch
    rng = np.random.default_rng(19)
    B, N, H, G, D, P, V = 4, 12, 2, 2, 64, 16, 50
    prompt = [0, 9, 16, 40]
    c, table = kh.make_cache(rng, "e4m3", [0] * B, P, H, D, extra=40 + 4 * N, poison=False)
    dev, tab = kh.to_device(gpu_lib, c), _i32(table)
    (k, k64), (v, v64) = _rand(rng, (B, 40, H, D), "bf16"), _rand(rng, (B, 40, H, D), "bf16")
    cur = gpu_lib.kv_append(dev, tab, k, v, _i32([0] * B), counts=_i32(prompt))
    lens = okv.append(c, table, k64, v64, [0] * B, prompt)
    head = torch.from_numpy(rng.normal(size=(H * G * D, V)).astype(np.float32)).cuda()
    for _ in range(3):
        par = _tree(rng, B, N)
        (q, q64), (k, k64), (v, v64) = (_rand(rng, (B, N, h, D), "bf16") for h in (H * G, H, H))
        out, _ = _check_attention(gpu_lib, c, table, lens, (q, q64), (k, k64), (v, v64), D ** -0.5, "bf16", par,
                                  dev=dev)
        logits = (out.float().view(B, N, -1) @ head).contiguous()
        tok = np.zeros((B, N), np.int32)
        arg = logits.argmax(-1).cpu().numpy()
        for b in range(B):  # half of the nodes propose the target's choice after their parent
            for n in range(1, N):
                tok[b, n] = arg[b, par[b, n]] if rng.random() < 0.6 else (arg[b, par[b, n]] + 1) % V
        _, path, n_acc = gpu_lib.verify_tree_greedy(logits, _i32(tok), _i32(par))
        want = verify_tree_greedy(logits.cpu().numpy(), tok, par)
        np.testing.assert_array_equal(path.cpu().numpy(), want[1])
        cur = gpu_lib.kv_append(dev, tab, k, v, cur, index=path)
        lens = okv.append(c, table, k64, v64, lens, index=path.cpu().numpy())
        np.testing.assert_array_equal(cur.cpu().numpy(), lens)
        np.testing.assert_array_equal(n_acc.cpu().numpy() + 1 + np.asarray(prompt), lens)
        prompt = lens
        _same_cache(kh.to_host(dev, "e4m3"), c)
    kk, vv = gpu_lib.kv_read(dev, tab, cur, int(lens.max()))
    want = okv.read(c, table, lens, int(lens.max()))
    np.testing.assert_array_equal(kk.double().cpu().numpy(), want[0])
    np.testing.assert_array_equal(vv.double().cpu().numpy(), want[1])
