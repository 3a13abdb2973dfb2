"""Build libetg.so in-tree with hipcc for gfx950 (no JIT, no cache outside the repo)."""
from __future__ import annotations

import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libetg.so")
SOURCES = ["etg_api.cpp", "gather.hip", "logits.hip", "stream.hip", "wide.hip", "gemm.hip", "rank.hip", "q8.hip",
           "row.hip", "probe.hip", "quant.hip", "imatmul.hip", "sample.hip", "i8_sample_api.cpp",
           "xent.hip", "rowgrad.hip", "train_api.cpp", "noalloc.hip", "step.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17", "-Wall", "-Wno-unused-result",
    # keep packed-FP32 instructions out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]
# sources whose kernels must not spill registers: their waits count copies in flight, and what a spill
# adds to the count makes each wait one for more than it is meant for
NO_SPILLS = ("xent.hip",)


def spilled(remarks: str) -> list[str]:
    """Kernels with spilled vector registers in the compiler's resource remarks."""
    name, found = "", []
    for line in remarks.splitlines():
        m = re.search(r"remark:.*?(Function Name|VGPRs Spill): (\S+)", line)
        if m and m.group(1) == "Function Name":
            name = m.group(2)
        elif m and m.group(2) != "0":
            found.append(f"{name}: {m.group(2)}")
    return found


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    remarks = ["-Rpass-analysis=kernel-resource-usage"] if src in NO_SPILLS else []
    cmd = [HIPCC, *FLAGS, *remarks, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{out}")
    if remarks:
        if bad := spilled(out):
            raise RuntimeError(f"spilled vector registers in {src}: {'; '.join(bad)}")
        out = "\n".join(l for l in out.splitlines() if " warning: " in l)
    if out.strip():
        print(out, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source and link libetg.so next to this file.  Returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
