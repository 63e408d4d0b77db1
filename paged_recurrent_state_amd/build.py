"""Build libgdn_paged.so for gfx950 with hipcc (in-tree, no JIT cache).

Usage: python -m paged_recurrent_state_amd.build
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdn_paged.so")

SOURCES = ["gdn_slots.hip", "gdn_tables.hip", "gdn_check.hip", "gdn_prefill.hip", "gdn_decode.hip",
           "gdn_copy.hip", "gdn_rope.hip", "gdn_attention.hip", "gdn_api.hip"]

ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    # packed-FP32 instructions are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]

# Flags of single sources.
SOURCE_FLAGS = {
    # matrix products write to ordinary registers: the softmax works on the scores, and with the
    # accumulation registers as their destination every score is copied over first
    "gdn_attention.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
}


def hipcc() -> str:
    cand = os.environ.get("HIPCC") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(cand) and shutil.which(cand) is None:
        raise RuntimeError("hipcc not found (set HIPCC)")
    return cand


def spills(remarks: str) -> dict:
    """Kernels that keep vector registers in memory, from the compiler's resource remarks:
    {name: (registers spilled, bytes of scratch a lane)}."""
    found, name = {}, None
    for line in remarks.splitlines():
        m = re.search(r"remark:\s+(Function Name|VGPRs Spill|ScratchSize \[bytes/lane\]): (\S+)", line)
        if not m:
            continue
        if m[1] == "Function Name":
            name = m[2]
        elif int(m[2]):
            regs, scratch = found.get(name, (0, 0))
            found[name] = (int(m[2]), scratch) if m[1] == "VGPRs Spill" else (regs, int(m[2]))
    return found


def _compile(src: str, csrc: str = CSRC, objdir: str = OBJDIR) -> str:
    obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *FLAGS, *SOURCE_FLAGS.get(src, []), "-Rpass-analysis=kernel-resource-usage", "-I", INCLUDE,
           "-I", CSRC, "-c", os.path.join(csrc, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    # the kernels are laid out to fit the registers (the chunk attention's instances take up to 472 of 512):
    # one that no longer does is an error of its source, not only slower
    if bad := spills(r.stderr):
        os.remove(obj)
        raise RuntimeError(f"kernels of {src} spill (vector registers, bytes of scratch a lane): {bad}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link the shared library; returns its path."""
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), 8)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
