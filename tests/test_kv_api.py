"""The 8-bit cache's C ABI and binding without a GPU: sizes, refusals on the
host before any HIP call, and the same checks under AddressSanitizer."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import speculative_sampling_verify_spec_amd as sv
from speculative_sampling_verify_spec_amd import _kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_sampling_verify_spec_amd", "csrc")
F32, BF16 = sv.SPECV_F32, sv.SPECV_BF16
BASE = 0x10000  # fake device addresses: every call fails before it could touch them


@pytest.fixture(scope="module")
def lib():
    return sv.load()


class Kv(ctypes.Structure):
    """specv_kv_t."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "k_scales", "v_scales", "page_table")] + \
               [(n, ctypes.c_int) for n in ("num_pages", "max_pages", "page_size", "heads", "dim", "type")]


def kv(**kw):
    a = dict(k_pages=BASE, v_pages=2 * BASE, k_scales=3 * BASE, v_scales=4 * BASE, page_table=5 * BASE, num_pages=100,
             max_pages=10, page_size=64, heads=8, dim=128, type=sv.SPECV_E4M3)
    a.update(kw)
    return Kv(**a)


BAD_CACHE = [(dict(k_pages=None), -1), (dict(v_pages=None), -1), (dict(k_scales=None), -1), (dict(v_scales=None), -1),
             (dict(page_table=None), -1), (dict(type=2), -3), (dict(type=-1), -3), (dict(page_size=0), -2),
             (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=256), -2), (dict(num_pages=0), -2),
             (dict(max_pages=0), -2), (dict(max_pages=1 << 25), -2), (dict(heads=0), -2), (dict(heads=1 << 15), -2),
             (dict(dim=0), -2), (dict(dim=80), -2), (dict(dim=512), -2), (dict(k_pages=BASE + 8), -6),
             (dict(v_pages=BASE + 1), -6), (dict(k_scales=BASE + 2), -6)]


def append(lib, c=None, **kw):
    a = dict(k=6 * BASE, v=7 * BASE, row=0, lengths=8 * BASE, counts=None, index=None, B=4, N=3, out=None, dtype=BF16)
    a.update(kw)
    c = kv() if c is None else c
    return lib.spec_kv_append(ctypes.byref(c), a["k"], a["v"], a["row"], a["lengths"], a["counts"], a["index"], a["B"],
                              a["N"], a["out"], a["dtype"], None)


def read(lib, c=None, **kw):
    a = dict(starts=None, lengths=8 * BASE, B=4, T=3, k=6 * BASE, v=7 * BASE, dtype=BF16)
    a.update(kw)
    c = kv() if c is None else c
    return lib.spec_kv_read(ctypes.byref(c), a["starts"], a["lengths"], a["B"], a["T"], a["k"], a["v"], a["dtype"], None)


def attend(lib, c=None, **kw):
    a = dict(q=6 * BASE, qs=0, k=7 * BASE, v=8 * BASE, ks=0, lengths=9 * BASE, nodes=None, parents=None, scale=0.1, B=4,
             N=3, Hq=32, out=10 * BASE, lse=None, dtype=BF16, ws=16 * BASE, wsb=1 << 40)
    a.update(kw)
    c = kv() if c is None else c
    return lib.spec_kv_attention(ctypes.byref(c), a["q"], a["qs"], a["k"], a["v"], a["ks"], a["lengths"], a["nodes"],
                                 a["parents"], a["scale"], a["B"], a["N"], a["Hq"], a["out"], a["lse"], a["dtype"],
                                 a["ws"], a["wsb"], None)


def test_header_constants():
    text = open(os.path.join(ROOT, "include", "specverify.h")).read()
    assert re.search(r"SPECV_E4M3 = (\d+)", text).group(1) == str(sv.SPECV_E4M3)
    assert re.search(r"SPECV_I8 = (\d+)", text).group(1) == str(sv.SPECV_I8)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_caches(lib, kw, code):
    assert append(lib, kv(**kw)) == code
    assert read(lib, kv(**kw)) == code
    assert attend(lib, kv(**kw)) == code
    assert lib.spec_kv_attention_workspace_size(ctypes.byref(kv(**kw)), 4, 3, 32) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(k=None), -1), (dict(v=None), -1), (dict(lengths=None), -1), (dict(B=0), -2),
    (dict(B=65536), -2), (dict(N=0), -2), (dict(N=(1 << 24) + 1), -2), (dict(row=8 * 128 - 8), -2), (dict(row=-1), -2),
    (dict(row=8 * 128 + 4), -6), (dict(k=BASE + 8), -6), (dict(v=BASE + 4), -6)])
def test_append_refusals(lib, kw, code):
    assert append(lib, **kw) == code


def test_append_overlap(lib):
    """The new lengths may touch none of the arrays that other workgroups
    still read; right next to them is as far as they may go."""
    B, N, width = 4, 3, 10
    for name, at, n in (("lengths", 8 * BASE, B), ("counts", 10 * BASE, B), ("index", 11 * BASE, B * N),
                        ("page_table", 5 * BASE, B * width)):
        kw = {} if name == "page_table" else {name: at}
        for out in (at, at + 4, at - 4 * (B - 1), at + 4 * (n - 1)):
            assert append(lib, out=out, B=B, N=N, **kw) == -9, (name, out - at)
        for out in (at - 4 * B, at + 4 * n):
            assert append(lib, out=out, B=B, N=N, k=None, **kw) == -1
            assert append(lib, out=out, B=B, N=N, k=BASE + 8, **kw) == -6
    assert sv.ERRORS[-9] == "SPECV_E_OVERLAP" and "overlap" in sv.strerror(-9)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), -3), (dict(lengths=None), -1), (dict(k=None, v=None), -1), (dict(B=0), -2), (dict(T=0), -2),
    (dict(T=(1 << 24) + 1), -2), (dict(B=65536), -2), (dict(k=BASE + 8), -6), (dict(v=BASE + 8), -6)])
def test_read_refusals(lib, kw, code):
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), -3), (dict(q=None), -1), (dict(lengths=None), -1), (dict(out=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(B=0), -2), (dict(B=65536), -2), (dict(N=0), -2), (dict(N=65), -2), (dict(Hq=0), -2),
    (dict(Hq=12), -2), (dict(Hq=1 << 15), -2), (dict(Hq=8 * 1025), -2), (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(scale=-3.2e38), -2),
    (dict(qs=100), -2), (dict(qs=32 * 128 + 4), -6), (dict(ks=8 * 128 + 1), -6), (dict(q=BASE + 2), -6),
    (dict(k=BASE + 8), -6), (dict(v=BASE + 8), -6), (dict(out=BASE + 8), -6), (dict(ws=None), -5),
    (dict(ws=BASE + 16), -5), (dict(wsb=8), -5)])
def test_attention_refusals(lib, kw, code):
    assert attend(lib, **kw) == code


def test_null_descriptor(lib):
    assert lib.spec_kv_append(None, BASE, BASE, 0, BASE, None, None, 1, 1, None, BF16, None) == -1
    assert lib.spec_kv_read(None, None, BASE, 1, 1, BASE, BASE, BF16, None) == -1
    assert lib.spec_kv_attention_workspace_size(None, 1, 1, 8) == 0


def test_workspace_sizes(lib):
    """Every valid shape has a size, and it does not overflow at the largest ones."""
    for B, N, Hq, c in ((1, 1, 8, kv()), (256, 9, 32, kv()), (4096, 64, 64, kv(heads=8, dim=256)), (65535, 1, 8, kv()),
                        (1, 64, 8192, kv(heads=8, dim=256, max_pages=(1 << 24) - 1))):
        n = lib.spec_kv_attention_workspace_size(ctypes.byref(c), B, N, Hq)
        assert 0 < n < 1 << 46 and n % 256 == 0, (B, N, Hq, n)
    for B, N, Hq in ((0, 1, 8), (1, 0, 8), (1, 65, 8), (1, 1, 0), (1, 1, 9), (65536, 1, 8)):
        assert lib.spec_kv_attention_workspace_size(ctypes.byref(kv()), B, N, Hq) == 0


def test_largest_attention_calls(lib):
    """The limits that the header states: the last size inside has a
    workspace size in both types' plans, whatever the table, the first outside is refused."""
    def size(B, N, Hq, **kw):
        return lib.spec_kv_attention_workspace_size(ctypes.byref(kv(**kw)), B, N, Hq)
    for pages, P in ((1, 16), ((1 << 24) - 1, 128)):
        for dim in (64, 96, 128, 256):
            t = dict(max_pages=pages, page_size=P, dim=dim)
            assert size(1023, 64, 1024, heads=1, **t) > 0 and size(1024, 64, 1024, heads=1, **t) == 0
            assert size(32767, 1, 512, heads=512, **t) > 0
            assert size(1, 64, 32767, heads=32767, **t) > 0 and size(1, 1, 32768, heads=32767, **t) == 0
            assert size(8191, 1, 8192, heads=8, **t) > 0 and size(8192, 1, 8192, heads=8, **t) == 0
    assert size(32768, 1, 512, heads=512) == 0  # 2^24 workgroups
    assert attend(lib, kv(heads=1), B=1024, N=64, Hq=1024) == -2
    assert attend(lib, kv(heads=512), B=32768, N=1, Hq=512) == -2


def _parts(pages=4, h=2, p=16, d=64, dtype=torch.int8):
    return [torch.zeros(pages, h, p, d, dtype=dtype), torch.zeros(pages, h, d, p, dtype=dtype),
            torch.zeros(pages, h), torch.zeros(pages, h)]


def test_descriptor_is_the_headers_struct():
    c = sv.KVCache(*_parts())
    want = Kv(c.k_pages.data_ptr(), c.v_pages.data_ptr(), c.k_scales.data_ptr(), c.v_scales.data_ptr(), 4096, 4, 9, 16,
              2, 64, sv.SPECV_I8)
    assert _kv._descriptor(c, 4096, 9) == bytes(want)


def test_cache_checks():
    c = sv.KVCache(*_parts())
    assert (c.page_size, c.heads, c.dim) == (16, 2, 64)
    assert sv.KVCache.empty(3, 32, 1, 96, device="cpu").k_pages.dtype == torch.float8_e4m3fn
    for i, bad in ((0, torch.zeros(4, 2, 16, 64)), (0, torch.zeros(4, 2, 16, dtype=torch.int8)),
                   (0, torch.zeros(4, 2, 8, 64, dtype=torch.int8)), (0, torch.zeros(4, 2, 16, 80, dtype=torch.int8)),
                   (1, torch.zeros(4, 2, 16, 64, dtype=torch.int8)), (1, torch.zeros(4, 2, 64, 16, dtype=torch.uint8)),
                   (2, torch.zeros(4, 2, dtype=torch.float64)), (3, torch.zeros(4, 3)),
                   (1, torch.zeros(4, 2, 16, 64, dtype=torch.int8).transpose(2, 3)), (2, torch.zeros(2, 4).t())):
        parts = _parts()
        parts[i] = bad
        with pytest.raises((TypeError, ValueError)):
            sv.KVCache(*parts)


def test_host_tensors_are_refused():
    c = sv.KVCache(*_parts())
    tab, ln = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 3, 2, 64)
    for call in (lambda: sv.kv_append(c, tab, x, x, ln), lambda: sv.kv_read(c, tab, ln, 3),
                 lambda: sv.kv_attention(c, tab, x, ln, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_token_strides():
    f = _kv._token_stride
    x = torch.zeros(3, 5, 10, 64)
    assert f("x", x[:, :, :4], 4, 64) == 640 and f("x", x[:, :, 9:], 1, 64) == 640
    assert f("x", x[:, :1, :4], 4, 64) == 3200 and f("x", x[:1, :1, :4], 4, 64) == 256
    assert f("x", x[:1, 1:3, :4], 4, 64) == 640
    for bad in (x[:, :, ::2], x[:, :3], x[..., ::2], x.transpose(1, 2), x[:, :1].expand(3, 5, 10, 64),
                x[:1, :1].expand(3, 1, 10, 64)):
        with pytest.raises(ValueError):
            f("x", bad, bad.shape[2], bad.shape[3])


def test_forward_only():
    """Results that follow inputs with gradients refuse a backward pass; their
    values, and results without such inputs, are left as they are."""
    _kv._bind_torch()
    out, lse = torch.randn(3, 4), torch.randn(3)
    a, b = torch.randn(2, requires_grad=True), torch.randn(2)
    assert _kv._forward_only((out, lse), (b, None, b)) == (out, lse)
    with torch.no_grad():
        assert _kv._forward_only((out, lse), (a, None, b)) == (out, lse)
    for inputs in ((a, None, None), (b, b, a)):
        given = (out.clone(), lse.clone())
        got = _kv._forward_only(given, inputs)
        assert all(torch.equal(g, t) and g.requires_grad and g is x for g, t, x in zip(got, (out, lse), given))
        for g in got:
            with pytest.raises(NotImplementedError, match="forward only"):
                (g.sum() + a.sum()).backward()
        got[0].mul_(2.0)  # in place, as results without gradients take it
        assert torch.equal(got[0], 2.0 * out)
        with pytest.raises(NotImplementedError, match="forward only"):
            got[0].sum().backward()
    assert a.grad is None


def test_build_finds_spills():
    from speculative_sampling_verify_spec_amd.build import _spills
    line = "k.hip:3:1: remark: {} [-Rpass-analysis=kernel-resource-usage]\n"
    text = line.format("Function Name: _Za") + line.format("    VGPRs: 12") + line.format("    VGPRs Spill: 0") + \
        line.format("Function Name: _Zb") + line.format("    SGPRs Spill: 4") + line.format("    VGPRs Spill: 7")
    assert _spills(text) == ["_Zb: 7 VGPRs"] and _spills("") == []


STUBS = """
#include "specverify.h"
#include "sv_kv.h"
namespace sv {
hipError_t launch_kv_append(const KvAppend&, int, int, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_kv_read(const KvRead&, int, int, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_kv_attention(const KvAttn&, int, int, hipStream_t) { return hipErrorInvalidValue; }
}
"""


PLAN_STUBS = """
#include "specverify.h"
#include "sv_kv.h"
namespace sv {
static KvAppend seen;
hipError_t launch_kv_append(const KvAppend& p, int, int, hipStream_t) { seen = p; return hipSuccess; }
hipError_t launch_kv_read(const KvRead&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_attention(const KvAttn&, int, int, hipStream_t) { return hipSuccess; }
}
extern "C" int groups() { return sv::seen.groups; }
extern "C" unsigned page_slots() { return sv::kv_slots(sv::seen.N, sv::seen.c.P); }
"""


def test_append_work_is_linear_in_the_tokens(tmp_path):
    """A workgroup of the append looks through the call's pages and indexes up
    to its own last one.  A head's workgroups look at no more than 1024 entries for each token, up to the longest call
    (with a workgroup for every page: 2^39 pages and 2^43 indexes)."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not found")
    stubs, so = tmp_path / "plan.cpp", tmp_path / "libkv_plan.so"
    stubs.write_text(PLAN_STUBS)
    r = subprocess.run([gxx, "-std=c++17", "-shared", "-fPIC", "-O1", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include",
                        os.path.join(CSRC, "api_kv.cpp"), str(stubs), "-o", str(so)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    plan = ctypes.CDLL(str(so))
    plan.spec_kv_append.argtypes = sv.load().spec_kv_append.argtypes
    for out in (8 * BASE - 16, 8 * BASE + 16, 5 * BASE + 160, 9 * BASE + 48):  # next to the arrays, not over them
        assert append(plan, counts=8 * BASE, index=9 * BASE, out=out) == 0
    for P in (16, 32, 64, 128):
        for N in (1, 2, P, P + 1, P + 2, 8191, 1 << 14, (1 << 14) + 17, 131072, 999999, 1 << 24):
            c = kv(page_size=P, max_pages=(1 << 24) // P + 2)
            assert plan.spec_kv_append(ctypes.byref(c), BASE, BASE, 0, BASE, None, BASE, 1, N, None, BF16, None) == 0
            groups, slots = plan.groups(), plan.page_slots()
            assert slots == (N + P - 2) // P + 1 and 1 <= groups <= slots
            per = -(-slots // groups)  # each takes an equal share
            pages = sum(min(slots, (g + 1) * per) for g in range(groups))
            indexes = sum(min(N, (g + 1) * per * P) for g in range(groups))
            assert pages <= 1024 * slots and indexes <= 1024 * N
            if 2 < slots <= 1024:
                assert per == 1  # nothing is taken in turns that can run at once


def test_host_checks_under_address_sanitizer(tmp_path):
    gxx = shutil.which("g++")
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip() \
        if gxx else ""
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("g++ or libasan not found")
    stubs, so = tmp_path / "stubs.cpp", tmp_path / "libkv_asan.so"
    stubs.write_text(STUBS)
    r = subprocess.run([gxx, "-std=c++17", "-shared", "-fPIC", "-g", "-O1", "-fsanitize=address", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include",
                        os.path.join(CSRC, "api_kv.cpp"), str(stubs), "-o", str(so)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "asan", "host_checks_kv.py"), str(so)],
                       capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and "host checks ok" in r.stdout, out[-4000:]
