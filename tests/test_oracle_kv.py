"""The 8-bit cache's oracle against torch's own formats and hand-made values (CPU)."""
import numpy as np
import pytest
import torch

from oracle import kv as okv


def test_e4m3_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(okv.decode(codes, "e4m3"), want)


def test_e4m3_rounding_is_torchs():
    rng = np.random.default_rng(0)
    tab = okv.decode(np.arange(127, dtype=np.uint8), "e4m3")
    mids = (tab[1:] + tab[:-1]) / 2
    y = np.concatenate([tab, mids, -mids, np.nextafter(mids, 1e9), np.nextafter(mids, 0),
                        rng.normal(size=5000) * np.exp2(rng.uniform(-12, 8, 5000)).astype(np.float64)])
    y = np.clip(y, -448, 448).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(okv.encode(y.astype(np.float64), "e4m3"), want)


def test_special_values():
    assert okv.encode(np.array([np.inf, -np.inf, np.nan]), "e4m3").tolist() == [0x7e, 0xfe, 0x7f]
    assert okv.encode(np.array([np.inf, -np.inf, np.nan]), "int8").view(np.int8).tolist() == [127, -127, 0]
    assert okv.encode(np.array([0.5, 1.5, 2.5, -0.5]), "int8").view(np.int8).tolist() == [0, 2, 2, 0]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales(fmt):
    top = okv.QMAX[fmt]
    assert okv.block_scale(np.array([0.0]), fmt) == 2.0 ** -126
    assert okv.block_scale(np.array([top, np.inf, np.nan]), fmt) == 1.0
    assert okv.block_scale(np.array([-np.nextafter(top, 1e9)]), fmt) == 2.0
    assert okv.block_scale(np.array([top / 1024]), fmt) == 2.0 ** -10


def _cache(pages, H, P, D, fmt):
    return dict(k_pages=np.zeros((pages, H, P, D), np.uint8), v_pages=np.zeros((pages, H, D, P), np.uint8),
                k_scales=np.zeros((pages, H), np.float32), v_scales=np.zeros((pages, H), np.float32), fmt=fmt)


def test_growth_rounds_the_old_codes_again():
    c = _cache(1, 1, 16, 64, "int8")
    tab = np.zeros((1, 1), np.int32)
    x = np.zeros((1, 1, 1, 64))
    x[0, 0, 0, :3] = [100.0, 3.0, 5.0]
    assert okv.append(c, tab, x, x, [0]).tolist() == [1]
    assert c["k_scales"][0, 0] == 1.0
    y = np.full((1, 1, 1, 64), 200.0)
    assert okv.append(c, tab, y, y, [1]).tolist() == [2]
    k, v = okv.read(c, tab, [2], 2)
    assert c["k_scales"][0, 0] == 2.0
    assert k[0, 0, 0, :4].tolist() == [100.0, 4.0, 4.0, 0.0]   # 1.5 and 2.5 round to even codes
    assert (k[0, 1] == 200.0).all() and (v == k).all()


def test_append_stops_at_bad_index_and_missing_page():
    c = _cache(3, 1, 16, 64, "e4m3")
    tab = np.array([[2, -1, 0], [1, 0, 7]], np.int32)
    x = np.ones((2, 20, 1, 64))
    assert okv.append(c, tab, x, x, [0, 16]).tolist() == [16, 32]
    idx = np.tile(np.arange(20), (2, 1))
    idx[0, 3], idx[1, 5] = -1, 20
    assert okv.append(c, tab, x, x, [0, 0], index=idx).tolist() == [3, 5]
    assert okv.append(c, tab, x, x, [0, 0], counts=[-4, 2]).tolist() == [0, 2]


def test_attention_of_nothing_and_of_one():
    c = _cache(1, 1, 16, 64, "e4m3")
    tab = np.zeros((1, 1), np.int32)
    q = np.ones((1, 2, 2, 64))
    out, lse, *_ = okv.attention(c, tab, q, [0], 0.5)
    assert (out == 0).all() and (lse == -np.inf).all()
    k = np.arange(2 * 64, dtype=float).reshape(1, 2, 1, 64)
    out, lse, *_ = okv.attention(c, tab, q, [0], 0.5, k, k)
    np.testing.assert_array_equal(out[0, 0], np.broadcast_to(k[0, 0], (2, 64)))
    np.testing.assert_allclose(lse[0, 0], 0.5 * k[0, 0].sum())


def test_node_sets():
    see = okv.node_sets([-1, 0, 0, 1, 1, 9, 2, -3], 8)
    assert see[3].tolist() == [1, 1, 0, 1, 0, 0, 0, 0] and see[5].sum() == 1 and see[7].sum() == 1
    assert (okv.node_sets(None, 3) == np.tril(np.ones((3, 3)))).all()
