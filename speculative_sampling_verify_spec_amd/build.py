"""Build libspecverify.so in-tree with hipcc for gfx950.

Usage: python -m speculative_sampling_verify_spec_amd.build [-v]
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libspecverify.so")
SOURCES = ["api.cpp", "k_sweep.hip", "k_rounds.hip", "k_verify.hip", "k_exact.hip", "k_short.hip", "k_greedy.hip", "k_stats.hip",
           "k_tree.hip", "k_ngram.hip", "k_ngram_map.hip", "k_validate.hip", "api_kv.cpp", "k_kv_cache.hip",
           "k_kv_attn_64.hip", "k_kv_attn_96.hip", "k_kv_attn_128.hip", "k_kv_attn_256.hip", "k_kv_join.hip",
           "api_prompt.cpp", "k_prompt_64.hip", "k_prompt_96.hip", "k_prompt_128.hip", "k_prompt_256.hip",
           "api_budget.cpp", "k_kv_weights.hip", "k_kv_evict.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-ffp-contract=fast",
         # packed fp32 instructions stay off: the compiler must not emit v_pk_*_f32
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Rpass-analysis=kernel-resource-usage",  # read by _spills
         "-Wall", "-Wno-unused-result", "-I", INCLUDE, "-I", CSRC]


def _spills(remarks: str) -> list:
    """Kernels of a compilation that spill vector registers to memory.  The
    compiler can reload a spilled register while lanes are still masked off, so
    that they keep another value: no kernel here may spill."""
    found, name = [], "?"
    for m in re.finditer(r"remark: (?:.*?)(Function Name|VGPRs Spill): (\S+)", remarks):
        if m[1] == "Function Name":
            name = m[2]
        elif int(m[2]):
            found.append(f"{name}: {m[2]} VGPRs")
    return found


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    spills = _spills(r.stderr)
    if spills:
        raise RuntimeError(f"{src}: kernels spill registers:\n" + "\n".join(spills))
    noise = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
    if verbose and noise:
        print("\n".join(noise), file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source and link the shared library; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", f"--offload-arch={ARCH}", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
