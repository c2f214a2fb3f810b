"""Builds libdeltalog.so (the C-ABI library) in-tree for sm_100a with nvcc.

    python -m linear_attention_recurrent_deltalog_b200.build [--force] [--ptxas-info]

Each .cu in csrc/ compiles to an object in _build/ (in parallel), then they
link into linear_attention_recurrent_deltalog_b200/libdeltalog.so with the CUDA
runtime linked statically, so the library depends on the driver only.
"""

from __future__ import annotations

import argparse
import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdeltalog.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


SCAN = "dl_ssm_tc.cu"


def start_registers() -> int:
    """Registers a thread of the scan's chunk kernel has to start with."""
    with open(os.path.join(CSRC, SCAN)) as f:
        return int(re.search(r"kStartRegs = (\d+)", f.read()).group(1))


def check_registers(ptxas: str) -> None:
    """Raises where the compiler gave a chunk kernel fewer registers than its roles share out (the
    launch refuses such a kernel, since its warps would wait for registers for good)."""
    need, name, seen = start_registers(), "", 0
    for line in ptxas.splitlines():
        if m := re.search(r"Compiling entry function '(\S+)'", line):
            name = m.group(1)
        elif "dl_ssm_chunk_kernel" in name and (m := re.search(r"Used (\d+) registers", line)):
            seen += 1
            if int(m.group(1)) < need:
                raise RuntimeError(f"{name}: {m.group(1)} registers a thread, its roles share out {need}")
    if seen == 0:
        raise RuntimeError(f"{SCAN}: no chunk kernel's registers in the compiler's output")


def _deps() -> list:
    return (glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, ptxas_info: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path."""
    if not force and not ptxas_info and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    procs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if ptxas_info or os.path.basename(src) == SCAN:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (p.returncode != 0 or ptxas_info or verbose):
            sys.stdout.write(out)
        if p.returncode != 0:
            failed.append(src)
        if os.path.basename(src) == SCAN:
            scan_out = out
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(f) for f in failed))
    check_registers(scan_out)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-lrt", "-ldl", "-lpthread"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills per kernel")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_info=a.ptxas_info, verbose=a.verbose))


if __name__ == "__main__":
    main()
