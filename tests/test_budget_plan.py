"""How the node weights are shared out over workgroups (CPU): api_budget.cpp with
launchers that only remember their plan."""
import ctypes
import os
import shutil
import subprocess

import pytest

import speculative_sampling_verify_spec_amd as sv
from test_kv_api import BASE, kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_sampling_verify_spec_amd", "csrc")

STUBS = r"""
#include "sv_budget.h"
namespace sv {
static unsigned last;
hipError_t launch_kv_weights(const KvWeights& p, int, int, hipStream_t) { last = p.splits; return hipSuccess; }
hipError_t launch_kv_evict(const KvEvict&, int, hipStream_t) { return hipSuccess; }
}  // namespace sv
extern "C" unsigned last_splits() { return sv::last; }
"""


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    gxx, tmp = shutil.which("g++"), tmp_path_factory.mktemp("plan")
    if not gxx:
        pytest.skip("no g++")
    stubs, so = tmp / "stubs.cpp", tmp / "libplan.so"
    stubs.write_text(STUBS)
    r = subprocess.run([gxx, "-std=c++17", "-shared", "-fPIC", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                        "-I", CSRC, "-I", "/opt/rocm/include", os.path.join(CSRC, "api_budget.cpp"), str(stubs), "-o", str(so)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    lib, far = ctypes.CDLL(str(so)), 1 << 44
    lib.spec_kv_weights.argtypes = sv.load().spec_kv_weights.argtypes

    def plan(B, heads, positions):
        c = kv(heads=heads, page_size=128, max_pages=positions // 128)
        rc = lib.spec_kv_weights(ctypes.byref(c), 6 * BASE, 0, 7 * BASE, None, 0, 9 * BASE, None, None, 0.1, B, 1, 4 * heads,
                                 far, far, positions, sv.SPECV_BF16, None)
        assert rc == 0
        return lib.last_splits()

    return plan


def test_long_tables_are_shared_at_any_number_of_pairs(splits):
    """One workgroup for a head of 32768 positions would be alone at the end,
    also where there are as many heads as fill the card with one each."""
    for pairs in range(1, 1024):
        n = splits(pairs, 1, 32768)
        assert n == splits(1, pairs, 32768)
        assert n * pairs <= 2048 and n >= min(512 // pairs, 128), (pairs, n)
        assert pairs < 128 or n * pairs >= 1024, (pairs, n)


def test_short_tables_take_no_more_than_they_have(splits):
    for pairs in (1, 3, 64, 511, 512, 513, 2000, 2049, 70000):
        for positions in (128, 256, 2048, 4096, 1 << 20):
            n = splits(pairs, 1, positions) if pairs < 65536 else splits(pairs // 8, 8, positions)
            turns = -(-positions // 256)
            assert 1 <= n <= turns and (n == 1 or n * pairs <= 2048)
            if turns >= 512:
                assert n == max(1, 2048 // pairs) or pairs <= 8
