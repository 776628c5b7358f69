"""Builds the C-ABI shared library librow_top_select.so for gfx950 with hipcc.

Run as ``python row_top_select_amd/build.py`` (or through
``__graft_entry__.build()``); the library is written next to this file.  It
is run by path, not as a module of the package, because importing the
package loads the library.
"""

from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "librow_top_select.so")
OBJDIR = os.path.join(HERE, "_build")
SOURCES = ["rts_api.cpp", "rts_topk_rows.hip", "rts_merge.hip", "rts_slots.hip",
           "rts_indexer.hip", "rts_latent.hip", "rts_blocks.hip", "rts_beam.hip", "rts_kv.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # Packed fp32 VALU forms are avoided on this target.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-parameter",
]

# Flags of single sources.  Matrix products start with their results in vector
# registers and move to accumulation registers only under pressure.  The other
# way round the indexer spends 2 of 6 vector instructions a product on copying
# results back, and the latent kernels, which hold 256 registers of sums beside
# 16 of scores, push sums out to scratch (with it the widest one over listed rows
# still keeps one other register there).
_VECTOR_RESULTS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
EXTRA = {"rts_latent.hip": _VECTOR_RESULTS, "rts_indexer.hip": _VECTOR_RESULTS, "rts_kv.hip": _VECTOR_RESULTS}


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    err = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l)
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc link failed")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
