"""Loads from memory straight to LDS, in the assembly that the compiler makes
of the sources (CPU): the hardware takes their place in LDS from M0, and wants a
wait state between a scalar write of M0 and such a load.  The compiler places it
where it writes both itself, and not inside an inline assembly string."""
import os
import re
import shutil
import subprocess

import pytest

from speculative_sampling_verify_spec_amd import build

SOURCES = [s for s in build.SOURCES if s.startswith("k_prompt_")]


def hazards(asm):
    """(loads to LDS, those of them whose M0 was written by the instruction before)"""
    ins = [x for x in (re.sub(r"\s*(;|//).*", "", ln).strip() for ln in asm.splitlines())
           if x and not x.startswith(".") and not x.endswith(":")]
    loads = [i for i, x in enumerate(ins) if re.match(r"(global|buffer|scratch)_load_lds_|buffer_load_.* lds$", x)]
    return len(loads), [ins[i] for i in loads if i and re.match(r"s_\w+ m0\b", ins[i - 1])]


def test_what_counts():
    ok = "\ts_mov_b32 m0, s2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 v1, s[4:5]\n"
    bad = "k:\n\ts_add_i32 m0, s2, 4\n; a comment\n.L2:\n\tglobal_load_lds_dwordx4 v1, s[4:5] ; more\n"
    assert hazards(ok) == (1, []) and hazards(bad) == (1, ["global_load_lds_dwordx4 v1, s[4:5]"])


@pytest.mark.parametrize("src", SOURCES)
def test_a_wait_state_behind_writes_of_m0(tmp_path, src):
    if not (os.path.exists(build.HIPCC) or shutil.which(build.HIPCC)):
        pytest.skip("no hipcc")
    out = tmp_path / "k.s"
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", "-x", "hip", os.path.join(build.CSRC, src), "-o",
                        str(out)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    loads, bad = hazards(out.read_text())
    assert loads > 0 and not bad, (loads, len(bad), bad[:3])
