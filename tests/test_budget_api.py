"""The C ABI and binding of the cache under a budget without a GPU: refusals
on the host before any HIP call."""
import ctypes

import pytest
import torch

import speculative_sampling_verify_spec_amd as sv
from test_kv_api import BAD_CACHE, BASE, _parts, kv

F32, BF16 = sv.SPECV_F32, sv.SPECV_BF16
FAR = 1 << 40  # arrays between which nothing can overlap


@pytest.fixture(scope="module")
def lib():
    return sv.load()


def weigh(lib, c=None, **kw):
    a = dict(q=6 * BASE, qs=0, lse=7 * BASE, k=8 * BASE, ks=0, lengths=9 * BASE, counts=None, index=None, scale=0.1, B=4,
             N=3, Hq=32, w=FAR, out=2 * FAR, C=640, dtype=BF16)
    a.update(kw)
    c = kv() if c is None else c
    return lib.spec_kv_weights(ctypes.byref(c), a["q"], a["qs"], a["lse"], a["k"], a["ks"], a["lengths"], a["counts"],
                               a["index"], a["scale"], a["B"], a["N"], a["Hq"], a["w"], a["out"], a["C"], a["dtype"], None)


def evict(lib, c=None, **kw):
    a = dict(lengths=9 * BASE, w=FAR, C=640, new=10 * BASE, budget=100, recent=10, limit=200, B=4, table=11 * BASE,
             out_len=12 * BASE, out=2 * FAR, kept=3 * FAR, ws=16 * BASE, wsb=1 << 40)
    a.update(kw)
    c = kv() if c is None else c
    return lib.spec_kv_evict(ctypes.byref(c), a["lengths"], a["w"], a["C"], a["new"], a["budget"], a["recent"],
                             a["limit"], a["B"], a["table"], a["out_len"], a["out"], a["kept"], a["ws"],
                             a["wsb"], None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_caches(lib, kw, code):
    assert weigh(lib, kv(**kw)) == code
    assert evict(lib, kv(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(q=None), -1), (dict(lse=None), -1), (dict(lengths=None), -1), (dict(w=None), -1),
    (dict(out=None), -1), (dict(B=0), -2), (dict(B=65536), -2), (dict(N=0), -2), (dict(N=65), -2), (dict(Hq=0), -2),
    (dict(Hq=12), -2), (dict(Hq=1 << 15), -2), (dict(Hq=8 * 1025), -2), (dict(C=639), -2), (dict(C=1 << 31), -2),
    (dict(scale=float("nan")), -2), (dict(scale=-3.2e38), -2), (dict(qs=100), -2), (dict(qs=32 * 128 + 4), -6),
    (dict(ks=8 * 128 + 1), -6), (dict(q=BASE + 2), -6), (dict(k=BASE + 8), -6),
    (dict(out=FAR + 4), -9), (dict(out=FAR - 4), -9), (dict(out=FAR + 4 * (4 * 8 * 640 - 1)), -9)])
def test_weights_refusals(lib, kw, code):
    assert weigh(lib, **kw) == code


def test_weights_overlap(lib):
    """The weights written may touch nothing else that the call reads, at either end of it."""
    B, N, Hq, H, D, C, width = 4, 3, 32, 8, 128, 640, 10
    all_ = 4 * B * H * C
    sizes = dict(q=2 * (B * N * 5000 - 5000 + Hq * D), lse=4 * B * N * Hq, k=2 * (B * N * 2000 - 2000 + H * D), lengths=4 * B,
                 counts=4 * B, index=4 * B * N, w=all_)
    at = {n: (i + 3) * FAR for i, n in enumerate(sizes)}
    for n, size in sizes.items():
        edges = (at[n] + size - 4, at[n] - all_ + 4) + ((at[n],) if n != "w" else ())
        for out in edges:
            assert weigh(lib, **{**at, "out": out, "qs": 5000, "ks": 2000}) == -9, n
    cache = dict(page_table=4 * B * width, k_pages=100 * H * 64 * D, k_scales=4 * 100 * H)
    far = {n: (i + 20) * FAR for i, n in enumerate(("k_pages", "v_pages", "k_scales", "v_scales", "page_table"))}
    for n, size in cache.items():
        for out in (far[n], far[n] + size - 4, far[n] - all_ + 4):
            assert weigh(lib, kv(**far), **{**at, "out": out}) == -9, n


def test_weights_of_too_many_heads(lib):
    assert weigh(lib, kv(heads=512), B=32768, Hq=512) == -2


@pytest.mark.parametrize("kw,code", [
    (dict(lengths=None), -1), (dict(w=None), -1), (dict(new=None), -1), (dict(table=None), -1), (dict(out_len=None), -1),
    (dict(out=None), -1), (dict(kept=None), -1), (dict(B=0), -2), (dict(B=65536), -2), (dict(budget=0), -2),
    (dict(budget=641, limit=700), -2), (dict(recent=-1), -2), (dict(recent=101), -2), (dict(limit=99), -2),
    (dict(C=639), -2), (dict(C=1 << 31), -2), (dict(ws=None), -5), (dict(ws=BASE + 16), -5), (dict(wsb=255), -5)])
def test_evict_refusals(lib, kw, code):
    assert evict(lib, **kw) == code


def test_evict_overlap(lib):
    """An output may touch no input and no other output."""
    B, H, C, width, budget, new = 4, 8, 640, 10, 100, 2
    sizes = dict(lengths=B, w=B * H * C, new=B * new, table=B * width, out_len=B, out=B * H * C, kept=B * H * budget)
    at = dict(lengths=FAR, w=2 * FAR, new=3 * FAR, table=4 * FAR, out_len=5 * FAR, out=6 * FAR, kept=7 * FAR)
    for o in ("table", "out_len", "out", "kept"):
        for i in sizes:
            if i == o:
                continue
            for x in (at[i], at[i] + 4 * (sizes[i] - 1), at[i] - 4 * (sizes[o] - 1)):
                assert evict(lib, **{**at, o: x}) == -9, (o, i)
        for x in (5 * BASE, 5 * BASE + 4 * (B * width - 1)):  # the page table of kv()
            assert evict(lib, **{**at, o: x}) == -9, o


def test_evict_workspace_overlap(lib):
    """The workspace may touch no input and no output, at either end of it."""
    B, H, C, width, budget, new = 4, 8, 1 << 15, 257, 100, 2
    c = kv(max_pages=width)
    need = lib.spec_kv_evict_workspace_size(ctypes.byref(c), B)
    assert need == B * H * 2 * 16384
    sizes = dict(lengths=B, w=B * H * C, new=B * new, table=B * width, out_len=B, out=B * H * C, kept=B * H * budget)
    at = {n: (i + 2) * FAR for i, n in enumerate(sizes)}
    for n, size in sizes.items():
        for ws in (at[n], at[n] - need + 256, at[n] + (4 * size - 1) // 256 * 256):
            assert evict(lib, c, **{**at, "C": C, "ws": ws}) == -9, n


def test_evict_of_too_many_pages(lib):
    c = kv(heads=512, page_size=16, max_pages=1 << 15)
    far = {n: (i + 1) << 44 for i, n in enumerate(("lengths", "w", "new", "table", "out_len", "out", "kept"))}
    assert evict(lib, c, C=1 << 19, budget=1 << 19, limit=1 << 19, B=1, **far) == -2


def test_tables_of_next_to_2_31_positions(lib):
    """Positions are rounded up to whole workgroups in 32 bits, so the last 2^15 below 2^31 are refused."""
    most = ((1 << 31) - (1 << 15)) // 128
    for pages, ok in ((most, True), (most + 1, False), ((1 << 24) - 1, False)):
        c, C = kv(heads=1, page_size=128, max_pages=pages), (1 << 31) - 1
        assert (lib.spec_kv_evict_workspace_size(ctypes.byref(c), 1) > 0) == ok
        if not ok:
            far = {n: (i + 1) << 44 for i, n in enumerate(("lengths", "w", "new", "table", "out_len", "out", "kept"))}
            assert evict(lib, c, C=C, B=1, **far) == -2
            assert weigh(lib, c, C=C, B=1, Hq=4, w=FAR, out=FAR) == -2


def test_evict_workspace_sizes(lib):
    """256 bytes up to 16384 positions, then counts and lists of every 16384 of a head; 0 for what is refused."""
    def size(B, **kw):
        return lib.spec_kv_evict_workspace_size(ctypes.byref(kv(**kw)), B)
    assert size(4) == size(4, max_pages=256) == 256
    assert size(4, max_pages=257) == 4 * 8 * 2 * 16384 and size(1, heads=1, max_pages=1 << 24) == (1 << 16) * 16384
    assert size(0) == size(65536) == size(65535, heads=65) == size(4, max_pages=1 << 25) == 0
    assert lib.spec_kv_evict_workspace_size(None, 1) == 0
    far = {n: (i + 1) << 48 for i, n in enumerate(("lengths", "w", "new", "table", "out_len", "out", "kept"))}
    assert evict(lib, kv(max_pages=257), C=1 << 15, wsb=4 * 8 * 2 * 16384 - 1, **far) == -5
    assert evict(lib, kv(heads=65), B=65535, **far) == -2


def test_binding_refuses_host_tensors():
    c = sv.KVCache(*_parts())
    tab, ln = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x, lse, w = torch.zeros(1, 3, 2, 64), torch.zeros(1, 3, 2), torch.zeros(1, 2, 32)
    for call in (lambda: sv.kv_weights(c, tab, x, lse, ln, w), lambda: sv.kv_evict(c, tab, ln, w, tab[:, :1], 5, 1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
