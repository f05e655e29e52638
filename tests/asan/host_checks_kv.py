"""Host-side argument checks of the 8-bit cache, run against a CPU
AddressSanitizer build of api_kv.cpp (tests/test_kv_api.py builds it and runs
this file in a subprocess with libasan preloaded; no torch, no GPU).

usage: python host_checks_kv.py LIB.so"""
import ctypes
import sys

lib = ctypes.CDLL(sys.argv[1])
vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class Kv(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("k", "v", "ks", "vs", "table")] + \
               [(n, i32) for n in ("pages", "width", "P", "H", "D", "type")]


lib.spec_kv_append.argtypes = [vp, vp, vp, i64, vp, vp, vp, i32, i32, vp, i32, vp]
lib.spec_kv_read.argtypes = [vp, vp, vp, i32, i32, vp, vp, i32, vp]
lib.spec_kv_attention_workspace_size.argtypes = [vp, i32, i32, i32]
lib.spec_kv_attention_workspace_size.restype = sz
lib.spec_kv_attention.argtypes = [vp, vp, i64, vp, vp, i64, vp, vp, vp, f32, i32, i32, i32, vp, vp, i32, vp, sz, vp]
A = 0x10000
for P in (16, 32, 64, 128, 24):
    for D in (64, 96, 128, 256, 100):
        for fmt in (0, 1, 2):
            c = ctypes.byref(Kv(A, A, A, A, A, 7, 9, P, 4, D, fmt))
            ok = P != 24 and D != 100 and fmt != 2
            for dt in (0, 1, 3):
                want = -7 if ok and dt != 3 else None
                for B, N in ((1, 1), (300, 64)):
                    rcs = (lib.spec_kv_append(c, A, A, 0, A, None, None, B, N, None, dt, None),
                           lib.spec_kv_read(c, None, A, B, N, A, None, dt, None),
                           lib.spec_kv_attention(c, A, 0, A, A, 0, A, None, None, 1.0, B, N, 12, A, None, dt, A,
                                                 1 << 40, None))
                    assert all(r == want if want else r in (-2, -3) for r in rcs), (P, D, fmt, dt, rcs)
            for B, N, Hq in ((1, 1, 4), (4096, 64, 128), (0, 1, 4), (1, 65, 4), (1, 1, 5)):
                n = lib.spec_kv_attention_workspace_size(c, B, N, Hq)
                assert (n > 0) == (ok and B > 0 and N < 65 and Hq % 4 == 0)
print("host checks ok")
