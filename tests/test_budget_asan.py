"""The host side of whole prompts and of the cache under a budget
(api_prompt.cpp, api_budget.cpp) under AddressSanitizer, on the CPU, with
launchers that check what they are given: the multiplier that finds a row's
token, places for every block, workspaces that hold every tile."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_sampling_verify_spec_amd", "csrc")

STUBS = r"""
#include "sv_budget.h"
#include "sv_prompt.h"

namespace sv {
static hipError_t good(bool x) { return x ? hipSuccess : hipErrorInvalidValue; }

static bool packed(const Packed& s) {
  // rows at the steps from one token to the next, near the start and near 2^31
  for (long t0 : {0L, 1L, 77L, (1L << 31) / s.G - 2})
    for (long r = t0 * s.G; r < (t0 + 1) * s.G && r < (1L << 31); r += s.G > 1 ? s.G - 1 : 1) {
      const uint64_t y = s.G == 1 ? r : (static_cast<uint64_t>(r) * s.magic >> 32) >> s.shift;
      if (y != static_cast<uint64_t>(r / s.G)) return false;
    }
  return s.G * s.H == s.Hq && s.q_row > 0 && s.kv_row > 0 && s.q_row < (1 << 24) && s.kv_row < (1 << 24);
}
// B sequences of any lengths that add up to T take fewer places than there are
static hipError_t places(const Packed& s, unsigned slots, int per_token, int size) {
  const long one = (static_cast<long>(s.T) * per_token + size - 1) / size + (s.B - 1 < s.T ? s.B - 1 : s.T);
  return good(packed(s) && slots > one && static_cast<long>(slots) * s.H < (1L << 24) + s.H);
}
static hipError_t attn(const PromptAttn& p) { return places(p.s, p.slots, p.s.G, kPromptRows); }
static hipError_t weights(const PromptWeights& p) { return places(p.s, p.slots, 1, kWeightKeys); }
hipError_t launch_prompt_64(const PromptAttn& p, int, hipStream_t) { return attn(p); }
hipError_t launch_prompt_96(const PromptAttn& p, int, hipStream_t) { return attn(p); }
hipError_t launch_prompt_128(const PromptAttn& p, int, hipStream_t) { return attn(p); }
hipError_t launch_prompt_256(const PromptAttn& p, int, hipStream_t) { return attn(p); }
hipError_t launch_prompt_weights_64(const PromptWeights& p, int, hipStream_t) { return weights(p); }
hipError_t launch_prompt_weights_96(const PromptWeights& p, int, hipStream_t) { return weights(p); }
hipError_t launch_prompt_weights_128(const PromptWeights& p, int, hipStream_t) { return weights(p); }
hipError_t launch_prompt_weights_256(const PromptWeights& p, int, hipStream_t) { return weights(p); }
hipError_t launch_kv_weights(const KvWeights& p, int, int, hipStream_t) {
  const long positions = static_cast<long>(p.c.width) << p.c.pshift;
  return good(p.splits >= 1 && p.splits <= (positions + 255) / 256 && p.capacity >= positions);
}
hipError_t launch_kv_evict(const KvEvict& p, int, hipStream_t) {
  const long positions = static_cast<long>(p.c.width) << p.c.pshift;
  return good(static_cast<long>(p.tiles) * kEvictTile >= positions && (p.tiles - 1L) * kEvictTile < positions &&
              static_cast<long>(p.new_width) << p.c.pshift >= p.budget && p.limit >= p.budget);
}
}  // namespace sv
"""


def test_host_checks_under_address_sanitizer(tmp_path):
    gxx = shutil.which("g++")
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip() \
        if gxx else ""
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("g++ or libasan not found")
    stubs, so = tmp_path / "stubs.cpp", tmp_path / "libbudget_asan.so"
    stubs.write_text(STUBS)
    r = subprocess.run([gxx, "-std=c++17", "-shared", "-fPIC", "-g", "-O1", "-fsanitize=address", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include",
                        os.path.join(CSRC, "api_prompt.cpp"), os.path.join(CSRC, "api_budget.cpp"), str(stubs), "-o",
                        str(so)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "asan", "host_checks_budget.py"), str(so)],
                       capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out, out[-4000:]
    assert r.returncode == 0 and "host checks ok" in r.stdout, out[-4000:]
