"""Host-side argument checks and launch plans of whole prompts and of the cache
under a budget, run against a CPU AddressSanitizer build of api_prompt.cpp and
api_budget.cpp whose launchers check the plans they get
(tests/test_budget_asan.py builds it and runs this file in a subprocess with
libasan preloaded; no torch, no GPU).

usage: python host_checks_budget.py LIB.so"""
import ctypes
import sys

lib = ctypes.CDLL(sys.argv[1])
vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class Kv(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("k", "v", "ks", "vs", "table")] + \
               [(n, i32) for n in ("pages", "width", "P", "H", "D", "type")]


lib.spec_prompt_attention.argtypes = [vp, i64, vp, vp, i64, vp, f32, i32, i32, i32, i32, i32, vp, vp, i32, vp]
lib.spec_prompt_weights.argtypes = [vp, i64, vp, i64, vp, vp, f32, i32, i32, i32, i32, i32, vp, i64, i32, vp]
lib.spec_kv_weights.argtypes = [vp, vp, i64, vp, vp, i64, vp, vp, vp, f32, i32, i32, i32, vp, vp, i64, i32, vp]
lib.spec_kv_evict_workspace_size.argtypes = [vp, i32]
lib.spec_kv_evict_workspace_size.restype = sz
lib.spec_kv_evict.argtypes = [vp, vp, vp, i64, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
A, FAR = 0x10000, 1 << 44
OK, SHAPE, DTYPE, FORMAT = 0, -2, -3, -7  # a launcher that finds a fault in its plan gives SPECV_E_HIP

# ---- prompts: every group size, dims, strides ----
for heads, G in [(1, g) for g in range(1, 1025)] + [(8, 4), (3, 7), (128, 16), (32767, 1)]:
    Hq = heads * G
    want = OK if Hq <= 32767 and heads < 32768 else SHAPE
    assert lib.spec_prompt_attention(A, 0, A, A, 0, A, 0.1, 3, 100, heads, Hq, 64, A, None, 0, None) == want, (heads, G)
    assert lib.spec_prompt_weights(A, 0, A, 0, A, A, 0.1, 3, 100, heads, Hq, 64, A, 100, 1, None) == want, (heads, G)
for D in (64, 96, 128, 256, 100):
    for dt in (0, 1, 2):
        for B, T in ((1, 1), (65535, 1), (7, 1 << 24), (300, 100000), (0, 4), (2, 0)):
            want = DTYPE if dt == 2 else SHAPE if D == 100 or B == 0 or T == 0 else OK
            got = lib.spec_prompt_attention(A, 0, A, A, 0, A, 0.1, B, T, 2, 8, D, A, A, dt, None)
            assert got == want, (D, dt, B, T, got)
            got = lib.spec_prompt_weights(A, 0, A, 0, A, A, 0.1, B, T, 2, 8, D, A, 1 << 20, dt, None)
            assert got == want, (D, dt, B, T, got)
for stride, want in ((8 * 64, OK), (8 * 64 + 8, OK), ((1 << 24) - 8, OK), (1 << 24, SHAPE), (8 * 64 - 8, SHAPE)):
    assert lib.spec_prompt_attention(A, stride, A, A, 0, A, 0.1, 3, 100, 2, 8, 64, A, None, 1, None) == want, stride

# ---- the cache: every page size, dim and format; widths up to the largest ----
for P in (16, 32, 64, 128, 24):
    for D in (64, 96, 128, 256, 100):
        for fmt in (0, 1, 2):
            for width in (1, 9, 127, 129, 4096, 1 << 24):
                c = ctypes.byref(Kv(A, A, A, A, A, 7, width, P, 4, D, fmt))
                most = width * P
                ok = P != 24 and D != 100 and fmt != 2 and most < 1 << 31
                size = lib.spec_kv_evict_workspace_size(c, 3)
                if not ok:
                    assert size == 0
                for B, N in ((1, 1), (300, 64)):
                    got = lib.spec_kv_weights(c, A, 0, A, A, 0, A, None, None, 0.1, B, N, 12, FAR, FAR, min(most, 2 ** 31 - 1), 1, None)
                    assert (got == OK) == ok, (P, D, fmt, width, B, N, got)
                if not ok or not size:
                    continue
                for budget, recent, limit in ((1, 0, 1), (min(most, 130), 1, 1000), (min(most, 30000), 0, 1 << 30)):
                    for have, want in ((size, OK), (size - 1, -5)):
                        got = lib.spec_kv_evict(c, 1 * FAR, 2 * FAR, most, 3 * FAR, budget, recent, limit, 3, 4 * FAR,
                                                5 * FAR, 6 * FAR, 7 * FAR, A, have, None)
                        assert got == want, (P, D, fmt, width, budget, got)
print("host checks ok")
